"""Bounded waits of the state space scan's bf16 kernels that run out: with a
short limit, one hand-over between a kernel's warps is withheld, on which no copy
or product depends.  Each kernel must give up cleanly, record GDN2_ERR_TIMEOUT
and leave the context usable: the next call gives what the one before gave, bit
for bit.  (No fault, trap or endless wait is involved.)"""
import pytest
import torch

from test_gpu_ssm import GRADS, dev, make

pytestmark = pytest.mark.gpu


def short_of(g, chunk, call):
    """The status behind `call` with that chunk's hand-over withheld."""
    assert g.gdn2_get_device_status() == 0
    try:
        assert g.gdn2_debug_set(g.GDN2_DEBUG_WAIT_LIMIT, 1 << 12) == 0
        assert g.gdn2_debug_set(g.GDN2_DEBUG_WITHHOLD_READY, chunk) == 0
        call()
        return g.gdn2_get_device_status()
    finally:
        g.gdn2_debug_set(g.GDN2_DEBUG_WITHHOLD_READY, -1)
        g.gdn2_debug_set(g.GDN2_DEBUG_WAIT_LIMIT, 0)


def setup(T, H, dk, dv):
    import gated_delta_rule_gdn2_b200 as g
    d = dev(make(1, T, H, 1, dk, dv, "bf16", seed=131), "bf16")
    a = [d[n] for n in ("q", "k", "v", "la", "dt")]
    fwd = lambda: list(g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"]))  # noqa: E731

    def bwd():
        gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"])
        return [gr[n] for n in GRADS + ("dskip", "dS0")]

    return g, fwd, bwd


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("chunk", [0, 2, 3])
def test_forward(chunk, dk, dv):
    g, fwd, _ = setup(400, 2, dk, dv)
    want = fwd()
    assert short_of(g, chunk, fwd) == -4 and g.gdn2_get_device_status() == 0
    assert same(fwd(), want) and g.gdn2_get_device_status() == 0
    assert short_of(g, 4, fwd) == 0  # (no such chunk; the limit alone is long enough)


@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 64)])
def test_chains_of_states_and_gradients(dk, dv):
    """Three chunks; the backward's blocks have one unit each, of number 0."""
    g, _, bwd = setup(300, 1, dk, dv)
    want = bwd()
    for chunk in (1, 2):
        assert short_of(g, chunk, bwd) == -4 and g.gdn2_get_device_status() == 0
        assert same(bwd(), want) and g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_backward(dk, dv):
    """One chunk, whole or not; the second unit of each block."""
    for T in (128, 100):
        g, _, bwd = setup(T, 1, dk, dv)
        want = bwd()
        assert short_of(g, 1, bwd) == -4 and g.gdn2_get_device_status() == 0
        assert same(bwd(), want) and g.gdn2_get_device_status() == 0
        assert short_of(g, 2, bwd) == 0


@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 64)])
def test_parts_of_a_long_sequence(dk, dv):
    """A sequence cut into parts: their end states are left by a launch of their own."""
    g, fwd, bwd = setup(2048, 1, dk, dv)
    for call in (fwd, bwd):
        want = call()
        assert short_of(g, 1, call) == -4 and g.gdn2_get_device_status() == 0
        assert same(call(), want) and g.gdn2_get_device_status() == 0
