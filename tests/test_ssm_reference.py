"""The fp64 reference of the selective state space scan and its prologue,
against other forms of the same things, and the refusals of the C entry points
(which end before anything reaches the GPU)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn2_b200 as g
import ssm_ref as R

F64 = torch.float64


def _inputs(B, T, H, G, dk, dv, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    return dict(q=n(B, T, G, dk), k=n(B, T, G, dk), v=n(B, T, H, dv), la=-n(B, T, H).abs(), dt=n(B, T, H).abs(),
                skip=n(H), S0=n(B, H, dk, dv), dO=n(B, T, H, dv), dS_T=n(B, H, dk, dv))


def test_scan_is_the_masked_matrix_product():
    x = _inputs(2, 7, 4, 2, 3, 5)
    o, ST = R.scan(*[x[n] for n in ("q", "k", "v", "la", "dt", "skip", "S0")])
    L = x["la"].cumsum(1)
    for b in range(2):
        for h in range(4):
            q, k, v = x["q"][b, :, h // 2], x["k"][b, :, h // 2], x["v"][b, :, h]
            D = torch.exp(L[b, :, None, h] - L[b, None, :, h]).tril()
            want = ((q @ k.T) * D * x["dt"][b, None, :, h]) @ v + x["skip"][h] * v
            want = want + L[b, :, h].exp()[:, None] * (q @ x["S0"][b, h])
            torch.testing.assert_close(o[b, :, h], want, rtol=1e-12, atol=1e-12)
            w = torch.exp(L[b, -1, h] - L[b, :, h]) * x["dt"][b, :, h]
            torch.testing.assert_close(ST[b, h], L[b, -1, h].exp() * x["S0"][b, h] + (k * w[:, None]).T @ v, rtol=1e-12,
                                       atol=1e-12)


def test_scan_gradients_against_differences():
    x = _inputs(1, 5, 2, 1, 3, 2, seed=1)
    names = ("q", "k", "v", "la", "dt", "skip", "S0")
    gr = R.scan_grads(*[x[n] for n in names], x["dO"], x["dS_T"])

    def loss(y):
        o, ST = R.scan(*[y[n] for n in names])
        return float((o * x["dO"]).sum() + (ST * x["dS_T"]).sum())

    for n, gn in zip(names, ("dq", "dk", "dv", "dlog_alpha", "ddt", "dskip", "dS0")):
        for i in range(min(4, x[n].numel())):
            e = torch.zeros_like(x[n]).reshape(-1)
            e[(7 * i) % e.numel()] = 1e-6
            up, dn = dict(x), dict(x)
            up[n], dn[n] = x[n] + e.view_as(x[n]), x[n] - e.view_as(x[n])
            fd = (loss(up) - loss(dn)) / 2e-6
            assert abs(fd - float(gr[gn].reshape(-1)[(7 * i) % e.numel()])) <= 1e-6 * max(1.0, abs(fd)), n


def test_chunk_formulas_of_the_gradients():
    """The chunk form that the kernels compute (chunks of C tokens, E the
    gradient at a chunk's end), against autograd."""
    B, T, H, C = 1, 12, 1, 4
    x = _inputs(B, T, H, 1, 3, 5, seed=2)
    gr = R.scan_grads(*[x[n] for n in ("q", "k", "v", "la", "dt", "skip", "S0")], x["dO"], x["dS_T"])
    q, k, v, la, dt, dO = (x[n][0, :, 0] for n in ("q", "k", "v", "la", "dt", "dO"))
    S = [x["S0"][0, 0]]
    for t in range(T):
        S.append(la[t].exp() * S[-1] + dt[t] * torch.outer(k[t], v[t]))
    E = x["dS_T"][0, 0]
    out = {n: torch.zeros_like(y) for n, y in (("dq", q), ("dk", k), ("dv", v), ("dla", la), ("ddt", dt))}
    for c in range(T // C - 1, -1, -1):
        s = slice(c * C, (c + 1) * C)
        L = la[s].cumsum(0)
        D = torch.exp(L[:, None] - L[None]).tril()
        w = torch.exp(L[-1] - L)
        S0 = S[c * C]
        A = (q[s] @ k[s].T) * D
        Z = (dO[s] @ v[s].T) * D * dt[s][None]
        W = A * (dO[s] @ v[s].T) * dt[s][None]
        r = w * ((k[s] @ E) * v[s]).sum(1)
        u = L.exp() * ((q[s] @ S0) * dO[s]).sum(1)
        out["dv"][s] = dt[s][:, None] * (w[:, None] * (k[s] @ E) + A.T @ dO[s]) + x["skip"] * dO[s]
        out["dk"][s] = (dt[s] * w)[:, None] * (v[s] @ E.T) + Z.T @ q[s]
        out["dq"][s] = L.exp()[:, None] * (dO[s] @ S0.T) + Z @ k[s]
        out["ddt"][s] = r + (W / dt[s][None]).sum(0)
        low = W.tril(-1)
        run = (u + low.sum(1) - low.sum(0)).flip(0).cumsum(0).flip(0)
        out["dla"][s] = run + (dt[s] * r).cumsum(0) - dt[s] * r + L[-1].exp() * (E * S0).sum()
        E = L[-1].exp() * E + (q[s] * L.exp()[:, None]).T @ dO[s]
    for n, m in (("dq", "dq"), ("dk", "dk"), ("dv", "dv"), ("dla", "dlog_alpha"), ("ddt", "ddt")):
        torch.testing.assert_close(out[n], gr[m][0, :, 0], rtol=1e-11, atol=1e-11)
    torch.testing.assert_close(E, gr["dS0"][0, 0], rtol=1e-11, atol=1e-11)


def test_prologue_reference():
    gen = torch.Generator().manual_seed(3)
    x, W, b = (torch.randn(*s, generator=gen, dtype=F64) for s in ((6, 4), (4, 3), (4,)))
    init = torch.randn(2, 4, generator=gen, dtype=F64)
    xdt, dtb, A = (torch.randn(*s, generator=gen, dtype=F64) for s in ((6, 2), (2,), (2,)))
    y, dt, la, win = R.prologue(x, W, b, xdt, dtb, A, init)
    u = torch.nn.functional.conv1d(torch.cat([init, x]).T[None], W[:, None], b, groups=4)[0].T
    torch.testing.assert_close(y, torch.nn.functional.silu(u), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(dt, torch.nn.functional.softplus(xdt + dtb, threshold=50.), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(la, -A.exp() * dt)
    torch.testing.assert_close(win, x[-2:])
    # a sequence shorter than the window keeps part of the one before
    torch.testing.assert_close(R.prologue(x[:1], W, b, None, None, None, init)[3], torch.stack([init[1], x[0]]))


# ---------------------------------------------------------------------------
# refusals: (changed arguments, status)

P = 16
SCAN = dict(q=P, k=P, v=P, la=P, dt=P, skip=None, S0=None, o=P, S_T=None, states=None, cu=None, ldq=128, ldk=128,
            ldv=256, B=1, T=64, H=2, G=1, dk=128, dv=128, dtype=0, ws=P, ws_bytes=1 << 40)


def _fwd(**kw):
    return g.gdn2_ssm_fwd(*{**SCAN, **kw}.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=96), -2), (dict(dv=256), -2), (dict(dtype=2), -2), (dict(B=-1), -1), (dict(T=-1), -1), (dict(H=-1), -1),
    (dict(G=0), -1), (dict(H=3, G=2, ldv=384), -1), (dict(q=None), -1), (dict(k=24), -1), (dict(v=8), -1),
    (dict(o=None), -1), (dict(la=None), -1), (dict(la=17), -1), (dict(dt=17), -1), (dict(S0=8), -1), (dict(skip=18), -1),
    (dict(ldq=64), -1), (dict(ldk=132), -1), (dict(ldv=255), -1), (dict(ldv=260), -1), (dict(cu=18), -1),
    (dict(states=40), -1), (dict(B=1 << 20, H=64, ldv=8192), -1),
    (dict(H=1 << 24, ldv=1 << 31), -1), (dict(B=1 << 20, T=1 << 11), -1),
])
def test_scan_refuses(kw, code):
    assert _fwd(**kw) == code


def test_scan_workspace_refusals_and_empty_calls():
    n = g.gdn2_ssm_fwd_workspace(1, 32768, 2, 1, 128, 128, 1, 0)
    assert n > 0
    assert _fwd(T=32768, dtype=1, ws_bytes=n - 1) == -5 and _fwd(T=32768, dtype=1, ws=None, ws_bytes=0) == -5
    assert _fwd(B=0) == 0 and _fwd(H=0, G=1) == 0
    assert _fwd(T=0, S_T=None) == 0
    for q in (g.gdn2_ssm_fwd_workspace, lambda *a: g.gdn2_ssm_bwd_workspace(*a, 0)):
        assert q(0, 64, 2, 1, 128, 128, 0, 0) == 0 and q(1, 64, 2, 1, 96, 128, 0, 0) == 0
    assert g.gdn2_ssm_states_bytes(1, 64, 2, 96, 128, 0, 0) == 0
    # forming the states anew takes their room on top
    sizes = (3, 1000, 4, 2, 64, 128, 1, 1)
    assert g.gdn2_ssm_bwd_workspace(*sizes, 0) >= g.gdn2_ssm_bwd_workspace(*sizes, 1) + \
        g.gdn2_ssm_states_bytes(3, 1000, 4, 64, 128, 1, 1)


def _bwd(**kw):
    a = dict(q=P, k=P, v=P, la=P, dt=P, skip=None, S0=None, dO=P, dS_T=None, states=None, dq=P, dk_=P, dv_=P, dla=P,
             ddt=P, dskip=None, dS0=None, cu=None, ldq=128, ldk=128, ldv=256, B=1, T=64, H=2, G=1, dk=128, dv=128,
             dtype=0, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return g.gdn2_ssm_bwd(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=32), -2), (dict(dO=None), -1), (dict(dq=None), -1), (dict(dk_=24), -1), (dict(dv_=None), -1),
    (dict(dla=None), -1), (dict(ddt=17), -1), (dict(dS0=4), -1), (dict(dskip=18), -1), (dict(ws=None), -5),
    (dict(ws_bytes=64), -5), (dict(G=3), -1), (dict(ldv=128), -1), (dict(states=8), -1),
])
def test_scan_bwd_refuses(kw, code):
    assert _bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(S=None), -1), (dict(S=20), -1), (dict(o=None), -1), (dict(dk=80), -2), (dict(G=3), -1), (dict(ldq=127), -1),
    (dict(q=None), -1), (dict(dt=None), -1), (dict(B=-1), -1), (dict(B=0), 0), (dict(H=0), 0),
])
def test_step_refuses(kw, code):
    a = dict(q=P, k=P, v=P, la=P, dt=P, skip=None, S=P, o=P, ldq=128, ldk=128, ldv=256, B=1, H=2, G=1, dk=128, dv=128,
             dtype=0)
    a.update(kw)
    assert g.gdn2_ssm_step(*a.values(), 0) == code


PRO = dict(x=P, W=P, bias=None, K=4, xdt=P, dt_bias=None, A_log=P, init=None, y=P, dt=P, la=P, window=None, cu=None,
           ldx=64, ldt=2, B=1, T=8, C=64, H=2, dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), -2), (dict(K=5), -2), (dict(C=60), -2), (dict(dtype=3), -2), (dict(T=-1), -1), (dict(ldx=63), -1),
    (dict(ldt=1), -1), (dict(x=None), -1), (dict(x=17), -1), (dict(W=None), -1), (dict(W=6), -1), (dict(y=24), -1),
    (dict(init=8), -1), (dict(window=8), -1), (dict(xdt=None), -1), (dict(A_log=None), -1), (dict(dt=None), -1),
    (dict(cu=18), -1), (dict(bias=2), -1), (dict(B=0), 0), (dict(T=0), 0), (dict(C=0, H=0), 0),
    (dict(B=1 << 20, T=1 << 11), -1),
])
def test_prologue_refuses(kw, code):
    assert g.gdn2_ssm_prologue_fwd(*{**PRO, **kw}.values(), 0) == code


def test_prologue_bwd_and_step_refuse():
    def bwd(**kw):
        a = dict(x=P, W=P, bias=None, K=4, xdt=P, dt_bias=None, A_log=P, init=None, dy=P, ddt=P, dla=P, dx=P, dW=P,
                 dbias=None, dxdt=P, ddt_bias=None, dA_log=P, dinit=None, cu=None, ldx=64, ldt=2, B=1, T=8, C=64, H=2,
                 dtype=0, ws=P, ws_bytes=1 << 30)
        a.update(kw)
        return g.gdn2_ssm_prologue_bwd(*a.values(), 0)

    n = g.gdn2_ssm_prologue_bwd_workspace(1, 8, 64, 4, 2, 0)
    assert n == (64 * 5 + 4) * 4
    assert bwd(ws_bytes=n - 1) == -5 and bwd(ws=None) == -5 and bwd(K=5) == -2
    for m in ("x", "W", "dy", "ddt", "dla", "dx", "dW", "dxdt", "dA_log", "xdt", "A_log"):
        assert bwd(**{m: None}) == -1, m
    assert bwd(dinit=8) == -1 and bwd(dbias=2) == -1

    def step(**kw):
        a = dict(x=P, W=P, bias=None, K=4, xdt=P, dt_bias=None, A_log=P, window=P, y=P, dt=P, la=P, ldx=64, ldt=2, B=1,
                 C=64, H=2, dtype=0)
        a.update(kw)
        return g.gdn2_ssm_prologue_step(*a.values(), 0)

    assert step(window=None) == -1 and step(window=24) == -1 and step(x=None) == -1 and step(la=None) == -1
    assert step(B=0) == 0 and step(C=12) == -2


def test_torch_entry_points_check_their_tensors():
    x = torch.zeros(2, 8, 64)
    with pytest.raises((ValueError, TypeError)):  # host tensors
        g.ssm_prologue(x, torch.zeros(64, 4), None, None, None, None)
    q = torch.zeros(1, 4, 1, 64)
    v = torch.zeros(1, 4, 2, 64)
    with pytest.raises((ValueError, TypeError)):
        g.ssm_fwd(q, q, v, torch.zeros(1, 4, 2), torch.zeros(1, 4, 2))
    with pytest.raises(ValueError):  # groups that do not divide the heads
        g.ssm_fwd(q.expand(1, 4, 3, 64), q.expand(1, 4, 3, 64), v, torch.zeros(1, 4, 2), torch.zeros(1, 4, 2))
