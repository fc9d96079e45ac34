"""Calls of the state space operators that the entry points allow and the other
tests do not make."""
import pytest
import torch

import ssm_norms as N
import ssm_ref as R
from test_gpu_ssm import F64, GRADS, NAMES, SCAN, TD, check_all, cu_of, dev, make
from test_ssm_slices import slices

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_slices(dtype, packed):
    """q, k, v as slices of one tensor's rows, the gradients where the call puts
    them: as of contiguous copies, bit for bit."""
    import gated_delta_rule_gdn2_b200 as g
    H, G, dk, dv = 4, 2, 64, 128
    lens = (90, 0, 111) if packed else None
    d, cu = dev(make(3 if packed else 2, 201, H, G, dk, dv, dtype, lens=lens, seed=141), dtype), cu_of(lens)
    wide = torch.zeros(*d["v"].shape[:-2], H * dv + 2 * G * dk + 64, dtype=TD[dtype], device="cuda")
    views = slices(wide, H, G, dk, dv)
    for t, n in zip(views, "qkv"):
        t.copy_(d[n])
    rest = (d["la"], d["dt"], d["dO"])
    kw = dict(skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], cu_seqlens=cu)
    want = g.ssm_bwd(d["q"], d["k"], d["v"], *rest, **kw)
    before = torch.cuda.memory_allocated()
    got = g.ssm_bwd(*views, *rest, **kw)
    small = sum(got[n].numel() * got[n].element_size() for n in ("dlog_alpha", "ddt", "dskip", "dS0"))
    assert torch.cuda.memory_allocated() - before <= wide.numel() * wide.element_size() + small + (1 << 14)
    for n in GRADS + ("dskip", "dS0"):
        assert torch.equal(got[n], want[n]), n
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("T,dk,dv", [(16, 64, 64), (64, 128, 64), (150, 128, 128)])
def test_runs_of_resets(T, dk, dv, dtype):
    """Twelve resets in each run of sixteen tokens, as in front of a padded
    sequence's tokens: the four behind them see each other with all digits."""
    import gated_delta_rule_gdn2_b200 as g
    x = make(2, T, 2, 1, dk, dv, dtype, seed=151)
    at = torch.arange(T) % 16 < 12
    x["la"][:, at] = -1e4
    x["la"] = x["la"].to(TD[dtype]).to(F64)
    d = dev(x, dtype)
    check_all(x, d, dtype)
    ref = R.scan_grads(*[x[n] for n in NAMES], x["dO"], x["dS_T"])
    a = [d[n] for n in ("q", "k", "v", "la", "dt")]
    gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"])
    for n in GRADS:
        N.close(n, gr[n].cpu(), ref[n], N.BF16 if dtype == "bf16" else N.FP32, 2)


@pytest.mark.parametrize("B", [2, 150])
@pytest.mark.parametrize("T,dk,dv", [(1, 64, 128), (3, 128, 64), (100, 128, 128), (128, 64, 64)])
def test_heads_that_all_but_cancel(T, dk, dv, B):
    """Heads in pairs whose shares of dq and dk differ by a thirtieth or less:
    within a chunk without a state before it or a gradient behind, both are the sums of the heads'
    (v . dO) times k or q, and keep their digits, in one block and in one a head."""
    import gated_delta_rule_gdn2_b200 as g
    x = make(2, T, 16, 1, dk, dv, "bf16", s0=False, seed=161)
    near = 1 + 2.0 ** -5 * torch.rand(2, T, 8, dv, generator=torch.Generator().manual_seed(162), dtype=F64)
    for n in ("v", "dt", "la"):
        x[n][:, :, 1::2] = x[n][:, :, ::2]
    x["dO"][:, :, 1::2] = (-x["dO"][:, :, ::2] * near).to(torch.bfloat16).to(F64)
    d = {n: None if t is None or n in ("S0", "dS_T") else t if n == "skip" else t.repeat(B // 2, *[1] * (t.dim() - 1))
         for n, t in dev(x, "bf16").items()}
    gr = g.ssm_bwd(*[d[n] for n in ("q", "k", "v", "la", "dt")], d["dO"], skip=d["skip"])
    ref = R.scan_grads(*[x[n] for n in NAMES], x["dO"], x["dS_T"])
    for n in ("dq", "dk"):
        N.close(n, gr[n][:2].cpu(), ref[n], N.BF16, 2)
        assert torch.equal(gr[n], gr[n][:2].repeat(B // 2, 1, 1, 1))
