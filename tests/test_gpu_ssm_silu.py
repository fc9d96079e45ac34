"""The prologue's SiLU and its derivative over the whole range of their
argument: the convolution has one tap of weight 1, so u is x itself.

y = u s, s = 1 / (1 + e^{-u}): e^{-u} by the fast base-2 exponential has the
rounding of its argument, |u| 2^-24, and 2^-22 of its own; the reciprocal 2^-22;
under four roundings of 2^-24 besides: |y - ref| <= (|u| 2^-24 + 2^-20) |ref|
(for u > 0 less: e^{-u} is then the smaller part of the denominator; past |u| =
88 s is 0 or 1), and as s below 2^-126 may be 0, 128 2^-126 more.  The derivative
s (1 + u (1 - s)): the same of s (1 + |u| (1 - s)), 1 - s having s's error.
bf16: the result's rounding, 2^-8, and a result below the type's least normal."""
import pytest
import torch

from test_gpu_ssm import F64, TD

pytestmark = pytest.mark.gpu
LARGE = [39.0, 40.0, 57.0, 80.0, 87.0, 88.0, 100.0, 1e3, 1e6, 1e10, 1e15, 1e20, 1e30, 3e38]
ARGS = [0.0, 1e-30, 1e-3, 0.5, 1.0, 4.0, 16.0, 20.0, 30.0] + LARGE


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_silu_of_any_size(dtype):
    import gated_delta_rule_gdn2_b200 as g
    one = torch.tensor(ARGS + [-a for a in ARGS], dtype=F64)
    x = torch.cat([one.repeat_interleave(len(one)), one.repeat(len(one))]).view(2, -1).T.flatten()  # every pair side by side
    x = torch.nn.functional.pad(x, (0, -len(x) % 8)).to(TD[dtype]).to(F64)
    d, C = x.to("cuda", TD[dtype]), len(x)
    W, rows = torch.ones(C, 1, device="cuda"), d.view(1, 1, C).repeat(1, 3, 1)
    y = g.ssm_prologue(rows, W, None, None, None, None)[0]
    y1 = g.ssm_prologue_step(rows[:, 0], W, None, None, None, None, torch.empty(1, 0, C, dtype=TD[dtype], device="cuda"))[0]
    dx = g.ssm_prologue_bwd(rows, W, None, None, None, None, torch.ones_like(rows))["dx"]
    e = torch.exp(-x)
    s, n = 1 / (1 + e), 1 / (1 + torch.exp(x))
    rel = x.abs().clamp(max=104) * 2.0 ** -24 + 2.0 ** -20
    out = 2.0 ** -8 if dtype == "bf16" else 0.0
    for name, got, ref, mag in (("y", y, x * s, (x * s).abs()), ("token", y1, x * s, (x * s).abs()),
                                ("dx", dx, s * (1 + x * n), s * (1 + x.abs() * n))):
        err = (got.to(F64).cpu().reshape(-1, C) - ref).abs()
        ok = err <= rel * mag + out * ref.abs() + 128 * 2.0 ** -126
        at = (~ok).nonzero()
        assert bool(ok.all()), (name, [(float(x[j]), float(got.reshape(-1, C)[i, j]), float(ref[j])) for i, j in at[:5]])
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_nan_beside_a_number_stays_alone(dtype):
    import gated_delta_rule_gdn2_b200 as g
    x = torch.tensor([float("nan"), 2.0, -100.0, float("nan"), 1e20, float("nan"), float("inf"), 3.0], device="cuda").to(TD[dtype])
    W, rows = torch.ones(8, 1, device="cuda"), x.view(1, 1, 8)
    y = g.ssm_prologue(rows, W, None, None, None, None)[0].flatten()
    want = torch.nn.functional.silu(x.float())
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    keep = ~torch.isnan(want)
    torch.testing.assert_close(y[keep].float(), want[keep], rtol=2.0 ** -8, atol=1e-35)
