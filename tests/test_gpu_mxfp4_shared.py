"""The shared expert of the block served in 4 bits (test_gpu_mxfp4_block), stage by
stage: its quantised rows byte by byte, its activations against SiLU(gate) * up of
what those rows stand for, y against the product of the activations.  Then with
padding that is NaN: the other rows' bytes do not change."""
import pytest
import torch

import mxfp4_ref as ref
import test_gpu_ffn_mxfp4 as ffn
import test_gpu_mxfp4_block as blk

pytestmark = pytest.mark.gpu

N, H, I = blk.N, blk.H, blk.I


def _scales(t, cols):
    """[N, blocks], the short last tile's included."""
    return ref.take(t, N, -(-cols // 128) * 128)[0]


def _results(o):
    return [o["q"][0], _scales(o["s"], H), o["act"][0], _scales(o["act_scale"], I), o["y"][0]]


def test_shared_expert():
    import combine_moe_dispatch_gb300 as moe
    block = blk._Block(moe)
    o = block.own
    for seed in range(3):
        blk._inputs(80 + seed, block)
        padding = block.hidden.isnan().any(1)
        assert bool(padding.any())
        block.hidden[padding] = 0.25
        block.refill()
        block.forward()
        assert moe.read_status(block.b.workspace) == moe.Status.OK
        assert moe.read_status(block.shared_ws) == moe.Status.OK
        code, biased = ref.quantise(block.x)
        assert torch.equal(o["q"][0], ref.pack(code))
        assert torch.equal(_scales(o["s"], H), torch.nn.functional.pad(biased, (0, -(H // 32) % 4)))
        ffn._check(dict(o, c=[N], x=ref.values(code, biased)[None], wgu=block.shared["wgu"],
                        wd=block.shared["wd"]), 1, N, H, I)
        want = [t.clone() for t in _results(o)]
        block.hidden[padding] = float("nan")
        block.refill()
        block.forward()
        got = _results(o)
        for a, b in zip(want, got):
            assert torch.equal(a[~padding], b[~padding])
        assert bool((got[1][padding][:, :H // 32] == 255).all()) and bool(got[4][padding].isnan().all())
