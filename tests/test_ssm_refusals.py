"""More refusals of the state space entry points, before anything reaches the GPU."""
import pytest

import gated_delta_rule_gdn2_b200 as g

P = 16


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,T,code", [(2, 5, -1), (0, 5, 0), (2, 0, 0)])
def test_a_backward_without_heads_is_refused(B, T, code, dtype):
    """Nothing would write the gradients of q and k."""
    assert g.gdn2_ssm_bwd(P, P, P, P, P, None, None, P, None, None, P, P, P, P, P, None, None, None, 128, 128, 128, B, T, 0, 1,
                          128, 128, dtype, P, 1 << 20, 0) == code
