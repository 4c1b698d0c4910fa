"""moe_dispatch_mxfp4 with entries out of range, which set the status word while
other blocks begin: a bad entry is skipped, nothing outside the arrays and no row
that is not routed is touched, and a routed row's words are either the definition's
or, where a block saw the word already set, as they were.  One entry, and one
of every token of a batch that fills the GPU."""
import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

FILL = 0xA5
GUARD = 4096


def _guarded(dims):
    n = 1
    for d in dims:
        n *= d
    flat = torch.full((n + 2 * GUARD,), FILL, dtype=torch.uint8, device="cuda")
    return flat, flat[GUARD:GUARD + n].view(dims)


class _Call:
    def __init__(self, T, H, E, K, cap, seed):
        import combine_moe_dispatch_gb300 as moe
        self.moe, self.E, self.K, self.cap, self.H = moe, E, K, cap, H
        self.shape = moe.make_shape(1, T, H, E, K, cap)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
        self.idx = torch.rand((T, E), device="cuda", generator=g).argsort(1)[:, :K].int().contiguous()
        self.b = moe.Buffers(self.shape, expert_x=False, expert_y=False)
        self.flat_q, self.q = _guarded((E, cap, H // 2))
        self.flat_s, self.s = _guarded(tuple(ref.scale_tensor(E, cap, H, FILL).shape))

    def run(self, what, token, k, value):
        """Entries (token, k) get the value; returns the expected bytes and scales, and
        which rows may be written."""
        moe, b = self.moe, self.b
        b.plan(self.idx)
        assert moe.read_status(b.workspace) == moe.Status.OK
        self.flat_q.fill_(FILL)
        self.flat_s.fill_(FILL)
        i, s = self.idx.clone(), b.slot_of.clone()
        (i if what == "idx" else s)[token, k] = value
        good = torch.ones_like(i, dtype=torch.bool)
        good[token, k] = False
        moe.dispatch_mxfp4(self.shape, self.x, i, s, self.q, self.s, b.workspace)
        status = moe.read_status(b.workspace)
        rows = torch.zeros((self.E, self.cap, self.H), dtype=torch.bfloat16, device="cuda")
        below = torch.zeros((self.E, self.cap), dtype=torch.bool, device="cuda")
        at = i[good].long(), s[good].long()
        rows[at] = self.x[torch.arange(len(self.x), device="cuda")[:, None].expand(i.shape)[good]]
        below[at] = True
        return status, rows, below

    def check(self, rows, below):
        """Number of 16-byte words of the rows that were written."""
        code, biased = ref.quantise(rows)
        written = (self.q == ref.pack(code)).view(self.E, self.cap, -1, 16).all(-1)
        kept = (self.q == FILL).view(self.E, self.cap, -1, 16).all(-1)
        assert bool((written | kept)[below].all()) and bool(kept[~below].all())
        biased = torch.nn.functional.pad(biased, (0, -(self.H // 32) % 4))
        got = ref.take(self.s, self.cap, biased.shape[2] * 32)
        same = (got == biased).view(self.E, self.cap, -1, 4).all(-1)
        left = (got == FILL).view(self.E, self.cap, -1, 4).all(-1)
        assert bool((same | left)[below].all()) and bool(left[~below].all())
        # scale bytes that belong to no row
        rest = ref.place(torch.full_like(biased, FILL), self.s.clone())
        assert bool((rest == FILL).all())
        for flat in (self.flat_q, self.flat_s):
            assert bool((flat[:GUARD] == FILL).all()) and bool((flat[-GUARD:] == FILL).all())
        return int((written & ~kept)[below].sum())


@pytest.mark.parametrize("T,H,E,K,cap", [(64, 256, 8, 2, 64), (40, 1056, 5, 3, 40)])
def test_one_entry(T, H, E, K, cap):
    c = _Call(T, H, E, K, cap, 1)
    S = c.moe.Status
    for what, value, want in (("idx", E, S.BAD_EXPERT), ("idx", -2, S.BAD_EXPERT), ("idx", 1 << 30, S.BAD_EXPERT),
                              ("idx", -(1 << 31), S.BAD_EXPERT), ("slot", cap, S.CAPACITY), ("slot", -2, S.CAPACITY),
                              ("slot", (1 << 31) - 1, S.CAPACITY)):
        for token, k in ((0, 0), (9, K - 1), (T - 1, 0)):
            status, rows, below = c.run(what, token, k, value)
            assert status == want, (what, value)
            assert c.check(rows, below) > 0


def test_an_entry_of_every_token():
    """Words of the status race with its reading in every block: the call ends, and
    what it wrote is right."""
    T = 6000
    c = _Call(T, 1056, 16, 2, 1500, 2)
    for n in range(6):
        token = torch.arange(T, device="cuda")
        status, rows, below = c.run("idx" if n & 1 else "slot", token, n % 2, 1 << 20)
        assert status == (c.moe.Status.BAD_EXPERT if n & 1 else c.moe.Status.CAPACITY)
        assert c.check(rows, below) > 0
