"""Calls given a stream that is not the current one: what they allocate belongs
to that stream, so that work which the calling stream has pending cannot be
using the same memory."""
import types

import pytest
import torch

from test_gpu_ssm import dev, make, pro_inputs

pytestmark = pytest.mark.gpu


def tensors(x):
    if x is None:
        return []
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for y in (x.values() if isinstance(x, dict) else x) for t in tensors(y)]


def pool_of(t):
    """The stream whose memory pool holds t."""
    at = t.untyped_storage().data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds the tensor")


def ssm_calls(g):
    d = dev(make(2, 300, 4, 2, 128, 64, "bf16", seed=111), "bf16")
    a = [d[n] for n in ("q", "k", "v", "la", "dt")]
    one = [t[:, 0].contiguous() for t in a]
    _, _, p = pro_inputs((2, 70), 2, 64, 4, 3, "bf16", True, seed=112)
    w = [p[n] for n in ("W", "bias", "xdt", "dt_bias", "A_log")]
    first = [p["W"], p["bias"], p["xdt"][:, 0], p["dt_bias"], p["A_log"]]
    states = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True)[2]
    return {
        "ssm_fwd": lambda **k: g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True, **k),
        "ssm_bwd": lambda **k: g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=states, **k),
        "ssm_bwd, states anew": lambda **k: g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], **k),
        "ssm_step": lambda **k: g.ssm_step(*one, d["S0"].clone(), skip=d["skip"], **k),
        "ssm_prologue": lambda **k: g.ssm_prologue(p["x"], *w, init=p["init"], output_window=True, **k),
        "ssm_prologue_bwd": lambda **k: g.ssm_prologue_bwd(p["x"], *w, p["dy"], p["ddt"], p["dla"], init=p["init"], **k),
        "ssm_prologue_step": lambda **k: g.ssm_prologue_step(p["x"][:, 0], *first, p["init"].clone(), **k),
    }


def mixer_calls(g):
    gen = torch.Generator().manual_seed(113)
    r = lambda *s: torch.randn(*s, generator=gen).to("cuda", torch.bfloat16)  # noqa: E731
    B, T, H, D = 2, 150, 2, 128
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)  # noqa: E731
    q, k, v, w, dO = unit(r(B, T, H, D)), unit(r(B, T, H, D)), r(B, T, H, D), r(B, T, H, D).sigmoid(), r(B, T, H, D)
    la, b, beta = -r(B, T, H, D).abs(), r(B, T, H, D).sigmoid(), r(B, T, H).sigmoid()
    S0 = 0.1 * torch.randn(B, H, D, D, generator=gen).cuda()
    x, x1 = (q, k, v, la, b, w), [t[:, 0].contiguous() for t in (q, k, v, la, b, w)]
    cu = torch.tensor([0, 40, B * T], dtype=torch.int32, device="cuda")
    flat = [t.flatten(0, 1) for t in x]
    W, gamma = [torch.randn(H * D, 4, generator=gen).cuda() for _ in range(3)], torch.ones(D, device="cuda")
    states, fstates = g.chunk_fwd(*x, S0, save_states=True)[2], g.chunk_fwd_varlen(*flat, cu, S0, save_states=True)[2]
    grads = {"d" + n: t for n, t in zip(("q", "k", "v", "log_alpha", "b", "w"), (dO,) * 6)}
    return {
        "chunk_fwd": lambda **s: g.chunk_fwd(*x, S0, save_states=True, **s),
        "chunk_bwd": lambda **s: g.chunk_bwd(*x, S0, dO, **s),
        "chunk_bwd, states": lambda **s: g.chunk_bwd(*x, S0, dO, states=states, **s),
        "decode_step": lambda **s: g.decode_step(*x1, S0.clone(), **s),
        "chunk_fwd_varlen": lambda **s: g.chunk_fwd_varlen(*flat, cu, S0, save_states=True, **s),
        "chunk_bwd_varlen": lambda **s: g.chunk_bwd_varlen(*flat, cu, S0, dO.flatten(0, 1), states=fstates, **s),
        "chunk_fwd_reduced": lambda **s: g.chunk_fwd_reduced(q, k, v, la, beta, S0=S0, **s),
        "chunk_bwd_reduced": lambda **s: g.chunk_bwd_reduced(q, k, v, la, beta, S0, dO, **s),
        "decode_step_reduced": lambda **s: g.decode_step_reduced(*x1[:4], beta[:, 0].contiguous(), S0.clone(), **s),
        "prologue": lambda **s: g.prologue(q, k, v, *W, la, b, w, **s),
        "prologue_bwd": lambda **s: g.prologue_bwd(q, k, v, *W, la, b, w, grads, **s),
        "output_gate": lambda **s: g.output_gate(v, w, gamma, **s),
        "output_gate_bwd": lambda **s: g.output_gate_bwd(v, w, gamma, dO, **s),
        "chunk_fwd_gated": lambda **s: g.chunk_fwd_gated(*x, w, gamma, S0, **s),
    }


@pytest.mark.parametrize("calls", [ssm_calls, mixer_calls])
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_and_workspace_are_of_the_streams_pool(handle, calls, monkeypatch):
    import gated_delta_rule_gdn2_b200 as g
    from gated_delta_rule_gdn2_b200 import binding
    side, work = torch.cuda.Stream(), []
    scratch = binding._scratch

    def spy(*args):
        work.append(scratch(*args))
        return work[-1]

    monkeypatch.setattr(binding, "_scratch", spy)
    for name, call in calls(g).items():
        del work[:]
        torch.cuda.synchronize()
        out = tensors(call(stream=side.cuda_stream if handle else side))
        torch.cuda.synchronize()
        assert out
        for t in out + tensors(work):
            assert not t.numel() or pool_of(t) == side.cuda_stream, name
    assert torch.cuda.current_stream() != side and g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("make_calls", [ssm_calls, mixer_calls])
def test_a_call_elsewhere_right_behind_one_here(make_calls):
    """Without a wait between them, as often as not with what the call before
    has just given back."""
    import gated_delta_rule_gdn2_b200 as g
    calls = {n: f for n, f in make_calls(g).items() if "step" not in n}  # (those make their states on the current stream)
    want = {n: tensors(f()) for n, f in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        for n, f in calls.items():
            here = tensors(f())
            there = tensors(f(stream=side))
            f()
            torch.cuda.synchronize()
            for x, y, z in zip(want[n], here, there):
                assert torch.equal(x, y) and torch.equal(x, z), n


@pytest.mark.parametrize("calls", [ssm_calls, mixer_calls])
def test_a_stream_of_another_device_is_refused(calls):
    import gated_delta_rule_gdn2_b200 as g
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for n, f in calls(g).items():
        with pytest.raises(ValueError):
            f(stream=other)


@pytest.mark.parametrize("calls", [ssm_calls, mixer_calls])
def test_the_default_stream_by_its_handle(calls):
    """stream=0, with another stream current, and the current one by its own handle."""
    import gated_delta_rule_gdn2_b200 as g
    fs = {n: f for n, f in calls(g).items() if "step" not in n}  # (those make their states on the current stream)
    want = {n: tensors(f()) for n, f in fs.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for handle in (0, side.cuda_stream):
            for n, f in fs.items():
                out = tensors(f(stream=handle))
                torch.cuda.synchronize()
                for x, y in zip(want[n], out):
                    assert torch.equal(x, y), n
                    assert not y.numel() or pool_of(y) == handle, n
        assert torch.cuda.current_stream() == side
