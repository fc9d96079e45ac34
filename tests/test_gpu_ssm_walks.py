"""Walks of several chunks in the bf16 scan: what a chunk leaves in memory is
not touched by the chunks behind it."""
import pytest
import torch

from test_gpu_ssm import cu_of, dev, make

pytestmark = pytest.mark.gpu
TOKENS = ("q", "k", "v", "la", "dt")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dk,dv", [(64, 128), (64, 64), (128, 128), (128, 64)])
def test_a_chunks_rows_outlast_the_chunks_behind_it(dk, dv, packed):
    """The first rows of o do not depend on the tokens behind them: a call on T
    tokens gives, bit for bit, what calls on one chunk, two, .. of them give (no
    call is long enough to be cut into parts).  At dk < dv a block has one tile for
    the o of all its chunks."""
    import gated_delta_rule_gdn2_b200 as g
    B, H, T = 40, 8, 500
    d = dev(make(B, T, H, 2, dk, dv, "bf16", seed=101), "bf16")
    last = None
    for n in (128, 256, 300, 384, 499, 500):
        x = [d[m][:, :n].contiguous() for m in TOKENS]
        if packed:
            o, ST = g.ssm_fwd(*[t.flatten(0, 1) for t in x], skip=d["skip"], S0=d["S0"], cu_seqlens=cu_of([n] * B))
            o = o.view(B, n, H, dv)
        else:
            o, ST = g.ssm_fwd(*x, skip=d["skip"], S0=d["S0"])
        assert torch.isfinite(o).all() and torch.isfinite(ST).all()
        if last is not None:
            assert torch.equal(o[:, :last.shape[1]], last), n
        last = o
    assert g.gdn2_get_device_status() == 0
