"""The operators of a block served in 4 bits together, as a server calls them:
the residual's addition and the norm, the router, a plan of a ragged batch, the
dispatch that quantises, the experts on 4-bit operands, and the combine with a
shared expert, whose rows are quantised where they stand.  Eager, and captured
once and replayed with new inputs.

Each stage is checked against its definition on what the stage before it wrote:
the norm's rounding is bf16's half step and its sums' error (test_gpu_norm), the
4-bit rows are exact, the experts are checked as in test_gpu_ffn_mxfp4, and the
combine is one binary32 chain of K + 1 terms and one rounding."""
import pytest
import torch

import mxfp4_ref as ref
import test_gpu_ffn_mxfp4 as ffn

pytestmark = pytest.mark.gpu

D = torch.float64
R, T, H, I, E, K, CAP = 3, 40, 288, 160, 6, 2, 120
N, EPS = R * T, 1e-6


class _Block:
    def __init__(self, moe):
        self.moe = moe
        g = torch.Generator(device="cuda").manual_seed(50)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")

        def normal(*dims, std=1.0):
            return torch.empty(dims, **bf16).normal_(0.0, std, generator=g)

        self.shape = moe.make_shape(R, T, H, E, K, CAP)
        self.dense = moe.make_shape(1, N, H, 1, 1, N)
        self.b = moe.Buffers(self.shape, expert_x=False)
        self.b.workspace = torch.zeros(moe.ffn_mxfp4_workspace_size(self.shape, I), dtype=torch.uint8, device="cuda")
        self.shared_ws = torch.zeros(moe.ffn_mxfp4_workspace_size(self.dense, I), dtype=torch.uint8, device="cuda")
        self.gain, self.w_router = (1.0 + 0.1 * normal(H).float()).bfloat16(), normal(E, H, std=0.1).float()
        self.hidden, self.residual = normal(N, H), normal(N, H)
        self.sum, self.x, self.shared_y = (torch.empty((N, H), **bf16) for _ in range(3))
        self.num_tokens = torch.tensor([40, 0, 17], dtype=torch.int32, device="cuda")
        self.logits = torch.empty((N, E), device="cuda")
        self.idx = torch.empty((N, K), dtype=torch.int32, device="cuda")
        self.w = torch.empty((N, K), device="cuda")
        self.experts, self.shared = self._weights(E, normal), self._weights(1, normal)
        self.routed, self.own = self._rows(E, CAP), self._rows(1, N)

    def _weights(self, n, normal):
        """Quantised once, as a server does when it loads them."""
        moe, out = self.moe, {}
        for name, rows, cols, flags in (("wgu", 2 * I, H, moe.MXFP4_GATE_UP), ("wd", H, I, 0)):
            w = normal(n, rows, cols, std=cols ** -0.5)
            q = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
            s = torch.empty(moe.mxfp4_scale_bytes(n, rows, cols), dtype=torch.uint8, device="cuda")
            moe.quant_mxfp4(w, None, q, s, flags)
            code, biased = ref.quantise(w)
            assert torch.equal(q, ref.pack(code))
            out[name] = (q, s, ref.values(code, biased))
        return out

    def _rows(self, n, cap):
        u8 = dict(dtype=torch.uint8, device="cuda")
        return dict(q=torch.zeros((n, cap, H // 2), **u8), s=ref.scale_tensor(n, cap, H, 0),
                    act=torch.full((n, cap, I // 2), ffn.FILL, **u8), act_scale=ref.scale_tensor(n, cap, I, ffn.FILL),
                    y=torch.full((n, cap, H), ffn.SENTINEL, dtype=torch.bfloat16, device="cuda"))

    def forward(self):
        moe, b, r, o = self.moe, self.b, self.routed, self.own
        moe.add_rms_norm(self.shape, self.hidden, self.residual, self.gain, EPS, self.sum, self.x)
        torch.mm(self.x.float(), self.w_router.t(), out=self.logits)
        moe.router_topk(self.shape, self.logits, self.idx, self.w)
        b.plan_masked(self.idx, self.num_tokens)
        moe.dispatch_mxfp4(self.shape, self.x, self.idx, b.slot_of, r["q"], r["s"], b.workspace)
        w = self.experts
        moe.ffn_mxfp4(self.shape, I, r["q"], r["s"], *w["wgu"][:2], *w["wd"][:2], b.expert_num_tokens, r["act"],
                      r["act_scale"], r["y"], b.workspace)
        moe.quant_mxfp4(self.x[None], None, o["q"], o["s"])
        w = self.shared
        moe.ffn_mxfp4(self.dense, I, o["q"], o["s"], *w["wgu"][:2], *w["wd"][:2], None, o["act"], o["act_scale"],
                      o["y"], self.shared_ws)
        moe.combine_shared(self.shape, r["y"], self.idx, b.slot_of, self.w, o["y"], b.y, b.workspace)

    def refill(self):
        for rows in (self.routed, self.own):
            rows["act"].fill_(ffn.FILL)
            rows["act_scale"].fill_(ffn.FILL)
            rows["y"].fill_(ffn.SENTINEL)

    def check(self):
        b, moe = self.b, self.moe
        assert moe.read_status(b.workspace) == moe.Status.OK
        tokens = torch.arange(N, device="cuda")
        valid = tokens % T < self.num_tokens[tokens // T]
        s = (self.hidden.to(D) + self.residual.to(D)).bfloat16().to(D)
        assert torch.equal(self.sum[valid].to(D), s[valid])
        x = s * (s.square().mean(1, keepdim=True) + EPS).rsqrt() * self.gain.to(D)
        off = H * 2.0 ** -24 + 2.0 ** -20
        assert bool(((self.x.to(D) - x).abs() <= (2.0 ** -8 + off) * x.abs() + 2.0 ** -134)[valid].all())
        # the routed rows are the valid tokens', quantised
        code, biased = ref.quantise(self.x[valid])
        x4 = torch.zeros((N, H), dtype=D, device="cuda")
        x4[valid] = ref.values(code, biased)
        rows = torch.zeros((E, CAP, H), dtype=D, device="cuda")
        on = b.slot_of >= 0
        assert torch.equal(on.any(1), valid) and bool((on.all(1) == valid).all())
        token = tokens[:, None].expand(N, K)
        rows[self.idx[on].long(), b.slot_of[on].long()] = x4[token[on]]
        counts = torch.bincount(self.idx[on].long(), minlength=E)
        assert torch.equal(counts.int(), b.expert_num_tokens)
        for r, w, c, cap, x in ((self.routed, self.experts, counts.tolist(), CAP, rows),
                                (self.own, self.shared, None, N, x4[None])):
            if c is None:                    # every row exists: padding's are checked where they are finite
                for k in ("act", "y"):
                    r = dict(r, **{k: r[k][:, valid]})
                act = ref.values(ref.unpack(r["act"][0]), ref.take(r["act_scale"], N, I)[0][valid])
                y = act @ w["wd"][2][0].t()
                tol = 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * I * ffn.STEP * (act.abs() @ w["wd"][2][0].abs().t()) + 1e-30
                assert bool(((r["y"][0].to(D) - y).abs() <= tol).all())
                continue
            ffn._check(dict(r, c=c, x=x, wgu=w["wgu"], wd=w["wd"]), E, cap, H, I)
        total = self.own["y"][0].to(D).clone()
        size = total.abs()
        for k in range(K):
            t = tokens[on[:, k]]
            part = self.w[t, k, None].to(D) * self.routed["y"][self.idx[t, k].long(), b.slot_of[t, k].long()].to(D)
            total[t] += part
            size[t] += part.abs()
        tol = 2.0 ** -8 * total.abs() + 2 * K * ffn.STEP * size + 1e-30
        assert bool(((b.y.to(D) - total).abs() <= tol)[valid].all())


def _inputs(seed, block):
    g = torch.Generator(device="cuda").manual_seed(seed)
    block.hidden.normal_(0.0, 1.0, generator=g)
    block.residual.normal_(0.0, 3.0, generator=g)
    block.num_tokens.copy_(torch.randint(0, T + 1, (R,), generator=g, device="cuda"))
    tokens = torch.arange(N, device="cuda")
    block.hidden[tokens % T >= block.num_tokens[tokens // T]] = float("nan")       # padding


@pytest.mark.parametrize("graph", [False, True])
def test_block(graph):
    import combine_moe_dispatch_gb300 as moe
    block = _Block(moe)
    run = block.forward
    if graph:
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                block.forward()
        run = g.replay
    for seed in range(4):
        _inputs(60 + seed, block)
        block.refill()
        run()
        torch.cuda.synchronize()
        block.check()
