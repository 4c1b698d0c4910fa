"""Launches of moe_ffn and moe_ffn_backward back to back on one stream and one
workspace.  Each may start while the one before it drains, on the same SMs, with
barriers at the same places of shared memory: nothing of one launch may reach the
next.  (What a pair of CTAs sends to one another has to have arrived before either
leaves; a launch that broke this could pass all the same, so that this is a check of
the whole and not a proof.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


class _Call:
    """One shape's forward and backward pass into its own outputs."""

    def __init__(self, E, cap, H, I, counts, ws, seed):
        import combine_moe_dispatch_gb300 as moe
        self.moe, self.I, self.ws = moe, I, ws
        self.shape = moe.make_shape(1, E * cap, H, E, 1, cap)
        self.cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.x, self.dy = _normal((E, cap, H), 1.0, seed), _normal((E, cap, H), 1.0, seed + 1)
        self.h = _normal((E, cap, 2 * I), 1.0, seed + 2)
        self.wgu, self.wd = _normal((E, 2 * I, H), H ** -0.5, seed + 3), _normal((E, H, I), I ** -0.5, seed + 4)
        self.dims = [(E, cap, H), (E, cap, H), (E, 2 * I, H), (E, H, I)]
        self.act = torch.empty((E, cap, I), dtype=torch.bfloat16, device="cuda")
        self.dh = torch.empty((E, cap, 2 * I), dtype=torch.bfloat16, device="cuda")

    def outputs(self):
        return [torch.zeros(d, dtype=torch.bfloat16, device="cuda") for d in self.dims]

    def run(self, out):
        y, dx, dwgu, dwd = out
        self.moe.ffn(self.shape, self.I, self.x, self.wgu, self.wd, self.cnt, None, self.act, y, self.ws)
        self.moe.ffn_backward(self.shape, self.I, self.dy, self.x, self.h, self.wgu, self.wd, self.cnt,
                              self.act, self.dh, dx, dwgu, dwd, self.ws)


# no row at all, one tile, an empty expert, tokens over two tiles, a contraction that
# is cut, more experts than SM pairs
SHAPES = [(2, 4, 64, 64, [0, 0]), (1, 1, 8, 8, [1]), (3, 40, 264, 136, [40, 0, 7]),
          (1, 300, 136, 72, [290]), (3, 33, 1040, 2056, [33, 0, 7]), (90, 2, 64, 72, [1, 2, 0] * 30)]


@pytest.mark.parametrize("graph", [False, True])
def test_back_to_back(graph):
    import combine_moe_dispatch_gb300 as moe
    size = max(moe.ffn_workspace_size(moe.make_shape(1, E * cap, H, E, 1, cap), I)
               for E, cap, H, I, _ in SHAPES)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    calls = [_Call(*s, ws, 100 * i) for i, s in enumerate(SHAPES)]
    want = []
    for c in calls:                                # each alone
        out = c.outputs()
        torch.cuda.synchronize()
        c.run(out)
        torch.cuda.synchronize()
        want.append(out)
    order = [(7 * k + k // 6) % len(calls) for k in range(60)]
    got = [calls[i].outputs() for i in order]

    def all_of_them():
        for i, out in zip(order, got):
            calls[i].run(out)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_of_them()
    for _ in range(10):
        for out in got:
            for t in out:
                t.zero_()
        g.replay() if graph else all_of_them()
        for i, out in zip(order, got):
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), SHAPES[i]
    assert moe.read_status(ws) == moe.Status.OK
