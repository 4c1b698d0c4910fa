"""moe_ffn and moe_ffn_backward after a wait that ran out.  The failure is made
on the host, through words of the workspace's header (WsHeader in the kernels'
common header: the status in word 4, flags in word 5, the feed-forward's
counters from word 10 on); nothing faults or hangs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FLAGS, NEXT_UNIT = 5, 10              # 32-bit words of the header
BROKEN = -2 ** 31                     # bit 31 of the flags
SENTINEL = -12345.0


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


class _Step:
    """Plan and feed-forward of 12 tokens over 2 experts on one workspace."""

    def __init__(self):
        import combine_moe_dispatch_gb300 as moe
        self.moe, self.E, self.cap, self.H, self.I = moe, 2, 8, 128, 256
        E, cap, H, I = self.E, self.cap, self.H, self.I
        self.shape = moe.make_shape(1, 12, H, E, 1, cap)
        self.idx = torch.tensor([[i % 2] for i in range(12)], dtype=torch.int32, device="cuda")
        self.b = moe.Buffers(self.shape, expert_x=False, expert_y=False)
        self.ws = self.b.workspace = torch.zeros(moe.ffn_workspace_size(self.shape, I), dtype=torch.uint8,
                                                 device="cuda")
        self.x, self.dy = _normal((E, cap, H), 1.0, 1), _normal((E, cap, H), 1.0, 2)
        self.h = _normal((E, cap, 2 * I), 1.0, 3)
        self.wgu, self.wd = _normal((E, 2 * I, H), H ** -0.5, 4), _normal((E, H, I), I ** -0.5, 5)
        self.outs = [torch.empty(d, dtype=torch.bfloat16, device="cuda") for d in
                     ((E, cap, I), (E, cap, H), (E, cap, 2 * I), (E, cap, H), (E, 2 * I, H), (E, H, I))]

    def word(self, i, value):
        self.ws.view(torch.int32)[i] = value

    def plan(self):
        self.b.plan(self.idx)
        return self.moe.read_status(self.ws)

    def forward(self):
        act, y = self.outs[:2]
        self.moe.ffn(self.shape, self.I, self.x, self.wgu, self.wd, self.b.expert_num_tokens, None, act, y,
                     self.ws)
        return self.moe.read_status(self.ws)

    def backward(self):
        act, _, dh, dx, dwgu, dwd = self.outs
        self.moe.ffn_backward(self.shape, self.I, self.dy, self.x, self.h, self.wgu, self.wd,
                              self.b.expert_num_tokens, act, dh, dx, dwgu, dwd, self.ws)
        return self.moe.read_status(self.ws)

    def clear(self):
        for t in self.outs:
            t.fill_(SENTINEL)

    def untouched(self):
        return all(bool((t == SENTINEL).all()) for t in self.outs)

    def results(self):
        """Plan, forward and backward; what they write."""
        S = self.moe.Status
        self.clear()
        assert (self.plan(), self.forward(), self.backward()) == (S.OK, S.OK, S.OK)
        return [t.clone() for t in self.outs]

    def refuses(self):
        """After a plan that succeeds, each call reports TIMEOUT again and
        writes nothing, any number of times."""
        S = self.moe.Status
        for call in (self.forward, self.backward, self.forward, self.backward):
            self.clear()
            assert self.plan() == S.OK
            assert call() == S.TIMEOUT
            assert self.untouched()


def test_refused_until_the_workspace_is_initialised():
    """The mark that a wait which ran out leaves behind outlives the next
    plan's status and the test hooks; moe_workspace_init clears it."""
    s = _Step()
    want = s.results()
    s.word(FLAGS, BROKEN)
    s.refuses()
    s.moe.workspace_set_debug(s.ws, 0, 0)
    s.refuses()
    s.moe.workspace_init(s.ws)
    assert all(torch.equal(a, b) for a, b in zip(s.results(), want))


def test_wait_that_runs_out():
    """The launch's unit counter is set past the tiles of a (2 token tiles of 2
    feature tiles), so that nobody computes them and the two tiles of y wait, 20
    ms at most, for a count that nothing raises: the kernel returns, reports
    TIMEOUT and writes nothing, and so do later calls."""
    s = _Step()
    want = s.results()
    s.moe.workspace_set_debug(s.ws, 0, 20_000_000)
    s.clear()
    assert s.plan() == s.moe.Status.OK
    s.word(NEXT_UNIT, 4)
    assert s.forward() == s.moe.Status.TIMEOUT
    assert s.untouched()
    s.moe.workspace_set_debug(s.ws, 0, 0)
    s.refuses()
    s.moe.workspace_init(s.ws)
    assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
