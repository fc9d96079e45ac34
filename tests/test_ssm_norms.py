"""The 2-norm comparison of ssm_norms.py refuses gradients that are wrong in
ways which bounds from sums of magnitudes let through."""
import pytest
import torch

import ssm_norms as N
import ssm_ref as R
from test_gpu_ssm import GRADS, NAMES, make


@pytest.mark.parametrize("B,T,H,G,dk,dv", [(2, 100, 3, 1, 64, 64), (1, 200, 4, 2, 64, 128)])
def test_wrong_gradients_are_refused(B, T, H, G, dk, dv):
    x = make(B, T, H, G, dk, dv, "bf16", seed=7)
    ref = R.scan_grads(*[x[n] for n in NAMES], x["dO"], x["dS_T"])
    for n in GRADS:
        for wrong in (torch.zeros_like(ref[n]), -ref[n], 0.95 * ref[n], 1.05 * ref[n]):
            with pytest.raises(AssertionError):
                N.close(n, wrong, ref[n], N.BF16, 2)
        rounded = ref[n].to(torch.bfloat16)
        assert N.close(n, rounded, ref[n], N.BF16, 2) < 2.0 ** -8
    # one head's alone; a token's own write left out of ddt, and left in dlog_alpha
    one = ref["dv"].clone()
    one[:, :, 1] *= 0.95
    r = H // G
    own = (x["q"] * x["k"]).sum(-1).repeat_interleave(r, 2) * (x["dO"] * x["v"]).sum(-1)
    for n, wrong in (("dv", one), ("ddt", ref["ddt"] - own), ("dlog_alpha", ref["dlog_alpha"] + x["dt"] * own)):
        with pytest.raises(AssertionError):
            N.close(n, wrong, ref[n], N.BF16, 2)
