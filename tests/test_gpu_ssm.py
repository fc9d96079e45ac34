"""The selective state space scan, its backward and single token, and the
layer's prologue on the GPU, against the fp64 reference of ssm_ref.py (the
bounds are derived there; a test says what it adds).

Operands rounded to bf16 in one product of the bf16 kernels, at most: o: the
state or the masked q.k product (1), and the state once more where it crosses a
chunk (2); gradients: the gradient at a chunk's end or the state, and the decay
weight on the other factor (3).  A gradient that adds fp32 terms of one
rounded product each stays under the same count."""
import numpy as np
import pytest
import torch

import ssm_ref as R

pytestmark = pytest.mark.gpu
F64 = torch.float64
NAMES = ("q", "k", "v", "la", "dt", "skip", "S0")
GRADS = ("dq", "dk", "dv", "dlog_alpha", "ddt")
SCAN = ["fp32", "bf16"]  # element types of the scan
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(B, T, H, G, dk, dv, dtype, lens=None, s0=True, skip=True, seed=0, decay=1.0):
    """Host inputs (fp64 holding values of the dtype)."""
    gen = torch.Generator().manual_seed(seed + 7919 * T + B)
    rows = (B, T) if lens is None else (T,)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    r = lambda t: t.to(TD[dtype]).to(F64)  # noqa: E731
    A = torch.rand(H, generator=gen) * 15 + 1
    dt = torch.nn.functional.softplus(n(*rows, H) - 3)
    x = dict(q=r(n(*rows, G, dk)), k=r(n(*rows, G, dk)), v=r(n(*rows, H, dv)), la=r(-A * dt * decay), dt=r(dt),
             dO=r(n(*rows, H, dv)))
    x["skip"] = n(H).to(F64) if skip else None
    x["S0"] = n(B, H, dk, dv).to(F64) if s0 else None
    x["dS_T"] = n(B, H, dk, dv).to(F64) if s0 else None
    return x


def dev(x, dtype):
    out = {}
    for n, t in x.items():
        out[n] = None if t is None else t.to("cuda", torch.float32 if n in ("skip", "S0", "dS_T") else TD[dtype])
    return out


def cu_of(lens):
    return None if lens is None else torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


def host(t):
    return t.to(F64).cpu()


def rels(dtype, T, dk, dv, ops):
    """(relative bound of mag, of |ref|) of a token-dtype output, and of an fp32 one."""
    b = R.sums_bound(T, dk, dv)
    if dtype == "fp32":
        return (b, 0.0), (b, 0.0)
    return (ops * 2.0 ** -8 + b, 2.0 ** -8), (2.0 ** -16 + b, 0.0)


def check_all(x, d, dtype, lens=None, grads=True, save=True):
    import gated_delta_rule_gdn2_b200 as g
    cu = cu_of(lens)
    T = x["v"].shape[0 if lens is not None else 1]
    dk, dv = x["q"].shape[-1], x["v"].shape[-1]
    ref = R.scan_grads(*[x[n] for n in NAMES], x["dO"], x["dS_T"], lens)
    mag = R.magnitudes(*[x[n] for n in NAMES], x["dO"], x["dS_T"], lens)
    args = [d[n] for n in ("q", "k", "v", "la", "dt")]
    r = g.ssm_fwd(*args, skip=d["skip"], S0=d["S0"], save_states=save, cu_seqlens=cu)
    tok, f32 = rels(dtype, T, dk, dv, 2)
    R.within("o", host(r[0]), ref["o"], mag["o"], *tok)
    R.within("S_T", host(r[1]), ref["S_T"], mag["S_T"], *f32)
    if grads:
        gr = g.ssm_bwd(*args, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=r[2] if save else None,
                       need_dS0=d["S0"] is not None, cu_seqlens=cu)
        tok, f32 = rels(dtype, T, dk, dv, 3)
        for n in GRADS:
            R.within(n, host(gr[n]), ref[n], mag[n], *tok, mag["dla_sum"] if n == "dlog_alpha" else 0.0)
        rows = T if lens is not None else T * x["v"].shape[0]
        if d["skip"] is not None:  # exact products, rows * dv of them summed
            R.within("dskip", host(gr["dskip"]), ref["dskip"], mag["dskip"], (rows + dv) * 2.0 ** -24)
        if d["S0"] is not None:
            R.within("dS0", host(gr["dS0"]), ref["dS0"], mag["dS0"], *f32)
    assert g.gdn2_get_device_status() == 0
    return r


CASES = [  # B, T, H, G, dk, dv
    (1, 1, 1, 1, 64, 64), (2, 3, 2, 1, 128, 128), (1, 63, 3, 1, 64, 128), (2, 64, 2, 2, 128, 64),
    (1, 65, 4, 2, 128, 128), (1, 127, 2, 1, 64, 64), (2, 128, 4, 1, 128, 128), (1, 129, 2, 1, 128, 128),
    (1, 300, 8, 2, 64, 128), (3, 257, 6, 3, 128, 64), (1, 1100, 2, 1, 128, 128), (1, 1280, 1, 1, 64, 64),
]


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("B,T,H,G,dk,dv", CASES)
def test_scan_and_gradients(B, T, H, G, dk, dv, dtype):
    x = make(B, T, H, G, dk, dv, dtype)
    check_all(x, dev(x, dtype), dtype)


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("skip,s0,save", [(False, False, True), (True, False, False), (False, True, False)])
def test_optional_arguments(skip, s0, save, dtype):
    x = make(2, 150, 4, 2, 128, 64, dtype, skip=skip, s0=s0, seed=3)
    check_all(x, dev(x, dtype), dtype, save=save)


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("lens", [(5, 0, 130, 1, 64, 77), (0, 0), (1,), (128, 128, 1), (700, 3, 0), (0, 129)])
def test_packed(lens, dtype):
    x = make(len(lens), sum(lens), 4, 2, 128, 64, dtype, lens=lens, seed=5)
    if sum(lens) == 0:
        import gated_delta_rule_gdn2_b200 as g
        d = dev(x, dtype)
        o, ST = g.ssm_fwd(*[d[n] for n in ("q", "k", "v", "la", "dt")], skip=d["skip"], S0=d["S0"], cu_seqlens=cu_of(lens))
        assert torch.equal(ST, d["S0"]) and o.numel() == 0
        gr = g.ssm_bwd(*[d[n] for n in ("q", "k", "v", "la", "dt")], d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"],
                       cu_seqlens=cu_of(lens))
        assert torch.equal(gr["dS0"], d["dS_T"]) and float(gr["dskip"].abs().sum()) == 0
        return
    check_all(x, dev(x, dtype), dtype, lens=lens)


@pytest.mark.parametrize("dtype", SCAN)
def test_packed_matches_each_sequence_alone(dtype):
    """Bit for bit where the sequences are not cut into parts (bf16: under
    eight chunks of 128; fp32: one of 64)."""
    import gated_delta_rule_gdn2_b200 as g
    lens = (70, 129, 200) if dtype == "bf16" else (30, 64, 51)
    x = make(3, sum(lens), 2, 1, 64, 64, dtype, lens=lens, seed=8)
    d = dev(x, dtype)
    names = ("q", "k", "v", "la", "dt")
    o, ST = g.ssm_fwd(*[d[n] for n in names], skip=d["skip"], S0=d["S0"], cu_seqlens=cu_of(lens))
    r = 0
    for b, n in enumerate(lens):
        ob, Sb = g.ssm_fwd(*[d[m][None, r:r + n].contiguous() for m in names], skip=d["skip"],
                           S0=d["S0"][b:b + 1].contiguous())
        assert torch.equal(ob[0], o[r:r + n]) and torch.equal(Sb[0], ST[b])
        r += n


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("packed", [False, True])
def test_views_of_one_tensor(dtype, packed):
    """q, k, v as slices of the prologue's output, the gradients into one of
    its shape: equal, bit for bit, to contiguous copies; the gaps untouched."""
    import gated_delta_rule_gdn2_b200 as g
    H, G, dk, dv = 4, 2, 128, 64
    lens = (90, 0, 111) if packed else None
    x = make(3 if packed else 2, 201, H, G, dk, dv, dtype, lens=lens, seed=11)
    d, cu = dev(x, dtype), cu_of(lens)
    lead = d["v"].shape[:-2]
    wide = torch.full(lead + (H * dv + 2 * G * dk + 64,), 3.0, dtype=TD[dtype], device="cuda")
    cut = lambda w: (w[..., H * dv + G * dk:H * dv + 2 * G * dk].unflatten(-1, (G, dk)),  # noqa: E731
                     w[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)), w[..., :H * dv].unflatten(-1, (H, dv)))
    for view, n in zip(cut(wide), ("q", "k", "v")):
        view.copy_(d[n])
    a, b = [d[n] for n in ("q", "k", "v")], list(cut(wide))
    rest = [d["la"], d["dt"]]
    dwide = torch.full_like(wide, 7.0)
    outs = []
    for qkv, into in ((a, None), (b, cut(dwide))):
        o, ST, st = g.ssm_fwd(*qkv, *rest, skip=d["skip"], S0=d["S0"], save_states=True, cu_seqlens=cu)
        gr = g.ssm_bwd(*qkv, *rest, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st, cu_seqlens=cu, into=into)
        outs.append([o, ST] + [gr[n] for n in GRADS + ("dskip", "dS0")])
    for s, t in zip(*outs):
        assert torch.equal(s, t)
    assert torch.all(dwide[..., -64:] == 7.0)
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", SCAN)
def test_resets_and_steps_of_zero(dtype):
    """Resets (a log decay of -1e4), tokens without a decay, and steps dt = 0
    (the token writes nothing, but its ddt is the write's weight)."""
    x = make(1, 260, 2, 1, 128, 128, dtype, seed=13)
    x["la"][:, 40] = -1e4
    x["la"][:, 130] = -1e4
    x["la"][:, 131:190] = 0
    x["la"][:, 200:, 1] = -90.0
    x["dt"][:, 70:75] = 0
    x["la"] = x["la"].to(TD[dtype]).to(F64)
    check_all(x, dev(x, dtype), dtype)


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("T", [260, 2100])
def test_resets_of_every_size_are_one(T, dtype):
    """-inf and the type's lowest value, side by side too, give bit for bit
    what -1e4 gives, in whole sequences, in parts and for a token; a NaN is
    not mistaken for one."""
    import gated_delta_rule_gdn2_b200 as g
    d = dev(make(1, T, 2, 1, 64, 128, dtype, seed=14), dtype)
    lowest = torch.finfo(TD[dtype]).min
    at = [0, 3, 4, 5, 40, 63, 64, 127, 128, 200, 201, T - 1]

    def run(*values):
        la = d["la"].clone()
        la[:, at] = torch.tensor([values[i % len(values)] for i in range(len(at))], dtype=la.dtype, device="cuda")[None, :, None]
        a = [d["q"], d["k"], d["v"], la, d["dt"]]
        o, ST, st = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True)
        gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st)
        S = d["S0"].clone()
        o1 = g.ssm_step(*[t[:, 0].contiguous() for t in a], S, skip=d["skip"])
        return [o, ST, o1, S] + [gr[n] for n in GRADS + ("dskip", "dS0")]

    want = run(-1e4)
    for s, t in zip(run(-float("inf"), lowest), want):
        assert torch.equal(s, t)
    o, ST = run(-1e4, float("nan"))[:2]
    assert torch.isnan(o[:, 3:]).all() and torch.isnan(ST).all()
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", SCAN)
def test_neighbours_infinities_stay_out(dtype):
    """Packed: infinities and NaN in one sequence, and behind the last, reach
    no other; rows of no sequence are left as they were."""
    import gated_delta_rule_gdn2_b200 as g
    lens = (37, 90, 20)
    x = make(3, sum(lens) + 30, 2, 1, 64, 128, dtype, lens=lens + (30,), seed=17)
    bad = {n: t.clone() if t is not None else None for n, t in x.items()}
    for n in ("q", "k", "v", "dO"):
        bad[n][37:127] = float("inf")
        bad[n][147:] = float("nan")
    for n in ("la", "dt"):
        bad[n][147:] = float("nan")
    d = dev(bad, dtype)
    cu = cu_of(lens)
    good = [i for i in range(147) if not 37 <= i < 127]
    ref = {}
    for b, s in ((0, slice(0, 37)), (2, slice(127, 147))):
        y = {n: x[n][None, s] for n in ("q", "k", "v", "la", "dt", "dO")}
        args = [y.get(n) if n in y else (x[n] if n == "skip" else x[n][b:b + 1]) for n in NAMES]
        ref[b] = (R.scan_grads(*args, y["dO"], x["dS_T"][b:b + 1]), R.magnitudes(*args, y["dO"], x["dS_T"][b:b + 1]), s)
    names = [d[n] for n in ("q", "k", "v", "la", "dt")]
    o, ST, st = g.ssm_fwd(*names, skip=d["skip"], S0=d["S0"], save_states=True, cu_seqlens=cu)
    into = tuple(torch.full_like(d[n], 5.0) for n in ("q", "k", "v"))
    gr = g.ssm_bwd(*names, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st, cu_seqlens=cu, into=into)
    tok, f32 = rels(dtype, 90, 64, 128, 3)
    for b, (r, m, s) in ref.items():
        R.within("o", host(o[s]), r["o"][0], m["o"][0], *tok)
        R.within("S_T", host(ST[b]), r["S_T"][0], m["S_T"][0], *f32)
        for n in GRADS:
            R.within(n, host(gr[n][s]), r[n][0], m[n][0], *tok, m["dla_sum"][0] if n == "dlog_alpha" else 0.0)
        R.within("dS0", host(gr["dS0"][b]), r["dS0"][0], m["dS0"][0], *f32)
    for t in into:
        assert torch.all(t[147:] == 5.0)
    assert len(good) == 57 and g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", SCAN)
def test_bad_offsets_are_skipped_and_recorded(dtype):
    import gated_delta_rule_gdn2_b200 as g
    x = make(3, 100, 2, 1, 64, 64, dtype, lens=(30, 40, 30), seed=19)
    d = dev(x, dtype)
    cu = torch.tensor([0, 30, 20, 4000], dtype=torch.int32, device="cuda")
    names = [d[n] for n in ("q", "k", "v", "la", "dt")]
    o, ST = g.ssm_fwd(*names, skip=d["skip"], S0=d["S0"], cu_seqlens=cu)
    assert g.gdn2_get_device_status() == -1
    good = cu_of((30, 0, 0))
    o2, ST2 = g.ssm_fwd(*names, skip=d["skip"], S0=d["S0"], cu_seqlens=good)
    assert torch.equal(o[:30], o2[:30]) and torch.equal(ST[0], ST2[0])
    g.ssm_bwd(*names, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], cu_seqlens=cu)
    assert g.gdn2_get_device_status() == -1
    W, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    xx = d["v"].reshape(100, 128)[:, :64]
    g.ssm_prologue(xx, W, b, None, None, None, cu_seqlens=cu)
    assert g.gdn2_get_device_status() == -1
    g.ssm_prologue_bwd(xx, W, b, None, None, None, xx.contiguous(), cu_seqlens=cu)
    assert g.gdn2_get_device_status() == -1


@pytest.mark.parametrize("dtype", SCAN)
def test_few_long_sequences_in_parts(dtype):
    """One long sequence is cut into parts: against the same tokens as a large
    batch would run them (prompts chained through S0), and repeatable."""
    import gated_delta_rule_gdn2_b200 as g
    x = make(1, 4100, 2, 1, 64, 64, dtype, seed=23, decay=0.02)
    d = dev(x, dtype)
    check_all(x, d, dtype)
    names = ("q", "k", "v", "la", "dt")
    a = g.ssm_fwd(*[d[n] for n in names], skip=d["skip"], S0=d["S0"])
    b = g.ssm_fwd(*[d[n] for n in names], skip=d["skip"], S0=d["S0"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", SCAN)
def test_gradients_repeat_bit_for_bit(dtype):
    import gated_delta_rule_gdn2_b200 as g
    x = make(2, 300, 8, 1, 128, 128, dtype, seed=29)
    d = dev(x, dtype)
    names = [d[n] for n in ("q", "k", "v", "la", "dt")]
    runs = []
    for _ in range(2):
        o, ST, st = g.ssm_fwd(*names, skip=d["skip"], S0=d["S0"], save_states=True)
        runs.append(g.ssm_bwd(*names, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st))
    for n in GRADS + ("dskip", "dS0"):
        assert torch.equal(runs[0][n], runs[1][n]), n


# ---------------------------------------------------------------------------
# one token


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,G,dk,dv", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 64), (2, 6, 3, 64, 128), (40, 16, 1, 128, 128)])
def test_step(B, H, G, dk, dv, dtype):
    import gated_delta_rule_gdn2_b200 as g
    x = make(B, 3, H, G, dk, dv, dtype, seed=31)
    d = dev(x, dtype)
    S = d["S0"].clone()
    for t in range(3):
        y = [d[n][:, t] for n in ("q", "k", "v")] + [d[n][:, t].contiguous() for n in ("la", "dt")]
        o = g.ssm_step(*y, S, skip=d["skip"])
        args = [x[n][:, :t + 1] for n in ("q", "k", "v", "la", "dt")]
        ro, rS = R.scan(*args, x["skip"], x["S0"])
        mo, mS = R.scan(*[a.abs() if i != 3 else a for i, a in enumerate(args)], x["skip"].abs(), x["S0"].abs())
        b = R.sums_bound(3, dk, dv)
        R.within("o", host(o), ro[:, t], mo[:, t], b, 2.0 ** -8 if dtype == "bf16" else 0.0)
        R.within("S", host(S), rS, mS, b)


# ---------------------------------------------------------------------------
# prologue


def pro_inputs(rows, B, C, K, H, dtype, init, bias=True, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    r = lambda t: t.to(TD[dtype]).to(F64)  # noqa: E731
    f = lambda t: t.to(torch.float32).to(F64)  # noqa: E731
    x = dict(x=r(n(*rows, C)), W=f(n(C, K) * 0.5), bias=f(n(C)) if bias else None, xdt=r(3 * n(*rows, H)) if H else None,
             dt_bias=f(n(H)) if H and bias else None, A_log=f(n(H)) if H else None,
             init=r(n(B, K - 1, C)) if init else None)
    up = dict(dy=r(n(*rows, C)), ddt=r(n(*rows, H)) if H else None, dla=r(n(*rows, H)) if H else None)
    d = {m: None if t is None else t.to("cuda", torch.float32 if m in ("W", "bias", "dt_bias", "A_log") else TD[dtype])
         for m, t in {**x, **up}.items()}
    if pad:  # rows of a wider tensor, at an odd offset
        wide = torch.zeros(*rows, C + H + pad, dtype=TD[dtype], device="cuda")
        wide[..., pad:pad + C] = d["x"]
        wide[..., pad + C:] = d["xdt"] if H else 0
        d["x"], d["xdt"] = wide[..., pad:pad + C], wide[..., pad + C:] if H else None
    return x, up, d


def check_prologue(x, up, d, dtype, lens=None):
    """Bounds: a result's rounding (2^-8 of bf16; fp32: within the rest) and
    2^-18 of the magnitudes: under 16 roundings of 2^-24 of a convolution's
    few terms and the fast exponential's 2^-20.  A parameter's gradient sums
    rows terms: rows 2^-24 more."""
    import gated_delta_rule_gdn2_b200 as g
    cu = cu_of(lens)
    K, rel = x["W"].shape[1], 2.0 ** -8 if dtype == "bf16" else 0.0
    w = [d[n] for n in ("W", "bias", "xdt", "dt_bias", "A_log")]
    y, dt, la, win = g.ssm_prologue(d["x"], *w, init=d["init"], output_window=True, cu_seqlens=cu)
    leaf = {n: None if t is None else t.clone().requires_grad_() for n, t in x.items()}
    order = ("x", "W", "bias", "xdt", "dt_bias", "A_log", "init")
    ry, rdt, rla, rwin = R.prologue_batch(*[leaf[n] for n in order], lens)
    n = ry.shape[0]  # packed: rows past the last sequence are not looked at
    u = R.prologue_batch(*[None if leaf[m] is None else leaf[m].detach().abs() for m in order], lens)
    R.within("y", host(y)[:n], ry.detach(), 1 + u[0], 2.0 ** -18, rel)
    assert torch.equal(host(win), rwin.detach())
    outs, ups = [ry], [up["dy"][:n]]
    if dt is not None:
        R.within("dt", host(dt)[:n], rdt.detach(), 1 + rdt.detach(), 2.0 ** -20, rel)
        R.within("la", host(la)[:n], rla.detach(), rla.detach().abs() + x["A_log"].exp(), 2.0 ** -20, rel)
        outs, ups = [ry, rdt, rla], ups + [up["ddt"][:n], up["dla"][:n]]
    have = [m for m in order if leaf[m] is not None and leaf[m].numel()]
    gr = dict(zip(have, torch.autograd.grad(outs, [leaf[m] for m in have], ups, allow_unused=True, materialize_grads=True)))
    got = g.ssm_prologue_bwd(d["x"], *w, d["dy"], d["ddt"], d["dla"], init=d["init"], cu_seqlens=cu)
    # magnitudes: |silu'| <= 1.1 with an error of 2^-19 (1 + |u|) absolute
    amp = 1.2 * up["dy"].abs() * (1 + (u[0].abs() if lens is None else torch.nn.functional.pad(u[0].abs(), (0, 0, 0, up["dy"].shape[0] - n))))
    lin = {m: None if leaf[m] is None else leaf[m].detach().abs().requires_grad_() for m in ("x", "W", "init")}

    def conv(xx, WW, ii):
        K1 = WW.shape[1] - 1
        seqs = list(range(xx.shape[0])) if lens is None else [slice(a, a + m) for a, m in
                                                              zip(np.cumsum([0] + list(lens[:-1])), lens)]
        tot = 0
        for b, s in enumerate(seqs):
            z = torch.cat([torch.zeros(K1, xx.shape[-1], dtype=F64) if ii is None else ii[b], xx[s]])
            for j in range(K1 + 1):
                tot = tot + (WW[:, j] * z[j:j + xx[s].shape[0]] * amp[s]).sum()
        return tot

    hv = [m for m in ("x", "W", "init") if lin[m] is not None and lin[m].numel()]
    mg = dict(zip(hv, torch.autograd.grad(conv(lin["x"], lin["W"], lin["init"]), [lin[m] for m in hv],
                                          allow_unused=True, materialize_grads=True)))
    rows = amp.numel() // amp.shape[-1]
    more = 2.0 ** -18 + rows * 2.0 ** -24
    R.within("dx", host(got["dx"])[:n] if lens is not None else host(got["dx"]), gr["x"][:n] if lens is not None else gr["x"],
             mg["x"][:n] if lens is not None else mg["x"], 2.0 ** -18, rel)
    R.within("dW", host(got["dW"]), gr["W"], mg["W"], more)
    if x["bias"] is not None:
        R.within("dbias", host(got["dbias"]), gr["bias"], amp.reshape(-1, amp.shape[-1]).sum(0), more)
    if "init" in hv:
        R.within("dinit", host(got["dinit"]), gr["init"], mg["init"], 2.0 ** -18, rel)
    if dt is not None:
        A = x["A_log"].exp()
        m = up["ddt"].abs() + A * up["dla"].abs()
        R.within("dxdt", host(got["dxdt"])[:n], gr["xdt"][:n], m[:n], 2.0 ** -18, rel)
        if x["dt_bias"] is not None:
            R.within("ddt_bias", host(got["ddt_bias"]), gr["dt_bias"], m.reshape(-1, m.shape[-1]).sum(0), more)
        mA = (A * up["dla"].abs()[:n] * (1 + rdt.detach())).reshape(-1, m.shape[-1]).sum(0)
        R.within("dA_log", host(got["dA_log"]), gr["A_log"], mA, more)
    assert g.gdn2_get_device_status() == 0
    return y, got


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,T,C,K,H,init,pad", [(1, 1, 8, 4, 1, True, 0), (2, 100, 64, 4, 3, True, 0),
                                                (3, 2, 136, 3, 16, True, 0), (2, 77, 2304, 2, 16, False, 64),
                                                (1, 300, 72, 1, 5, False, 0), (2, 65, 264, 4, 3, True, 3),
                                                (1, 40, 64, 4, 0, False, 1), (1, 1500, 640, 4, 300, True, 0)])
def test_prologue(B, T, C, K, H, init, pad, dtype):
    x, up, d = pro_inputs((B, T), B, C, K, H, dtype, init, seed=T + C, pad=pad)
    check_prologue(x, up, d, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [(5, 0, 64, 1, 2, 31, 0), (0, 0, 3), (1,), (200, 1, 1, 1, 33)])
@pytest.mark.parametrize("init", [False, True])
def test_prologue_packed(lens, init, dtype):
    x, up, d = pro_inputs((sum(lens),), len(lens), 72, 4, 3, dtype, init, bias=init, seed=len(lens))
    check_prologue(x, up, d, dtype, lens)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prologue_rows_of_no_sequence(dtype):
    """Behind the last sequence nothing is read or written, whatever lies there."""
    import gated_delta_rule_gdn2_b200 as g
    lens = (30, 0, 45)
    x, up, d = pro_inputs((75,), 3, 64, 4, 2, dtype, True, seed=41)
    _, want = check_prologue(x, up, d, dtype, lens)
    e = dict(d)
    for m in ("x", "xdt", "dy", "ddt", "dla"):
        e[m] = torch.cat([d[m], torch.full_like(d[m][:20], float("nan"))])
    outs = {"y": torch.full_like(e["x"], 9.0), "dt": torch.full_like(e["xdt"], 9.0), "la": torch.full_like(e["xdt"], 9.0)}
    cu = cu_of(lens)
    code = 0 if dtype == "bf16" else 1
    assert g.gdn2_ssm_prologue_fwd(e["x"], e["W"], e["bias"], 4, e["xdt"], e["dt_bias"], e["A_log"], e["init"], outs["y"],
                                   outs["dt"], outs["la"], None, cu, 64, 2, 3, 95, 64, 2, code) == 0
    for t in outs.values():
        assert torch.all(t[75:] == 9.0) and torch.all(torch.isfinite(t))
    got = g.ssm_prologue_bwd(e["x"], *[e[n] for n in ("W", "bias", "xdt", "dt_bias", "A_log")], e["dy"], e["ddt"], e["dla"],
                             init=e["init"], cu_seqlens=cu)
    for m in ("dW", "dbias", "ddt_bias", "dA_log", "dinit"):
        torch.testing.assert_close(got[m], want[m], rtol=1e-3 if dtype == "bf16" else 1e-5, atol=1e-4)
    assert torch.equal(got["dx"][:75], want["dx"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,C,H,pad", [(4, 264, 3, 0), (2, 64, 16, 3), (3, 2304, 0, 0), (1, 72, 2, 0)])
def test_prologue_step_continues_a_prompt(K, C, H, pad, dtype):
    """Tokens one by one give what the prompt gives, window included, bit for bit."""
    import gated_delta_rule_gdn2_b200 as g
    x, up, d = pro_inputs((3, 9), 3, C, K, H, dtype, K > 1, seed=K, pad=pad)
    w = [d[n] for n in ("W", "bias", "xdt", "dt_bias", "A_log")]
    y, dt, la, win = g.ssm_prologue(d["x"], *w, init=d["init"], output_window=True)
    window = torch.empty(3, 0, C, dtype=TD[dtype], device="cuda") if K == 1 else d["init"].clone()
    for t in range(9):
        ys, dts, las = g.ssm_prologue_step(d["x"][:, t], d["W"], d["bias"], None if not H else d["xdt"][:, t], d["dt_bias"],
                                           d["A_log"], window)
        assert torch.equal(ys, y[:, t])
        if H:
            assert torch.equal(dts, dt[:, t]) and torch.equal(las, la[:, t])
    assert torch.equal(window, win)


# ---------------------------------------------------------------------------
# as they are used together


def layer(g, p, proj, cfg, init=None, S0=None, cu=None, save=False):
    """in-projection [.., C + H] -> prologue -> scan -> output gate."""
    H, G, dk, dv = cfg
    C = H * dv + 2 * G * dk
    y, dt, la, win = g.ssm_prologue(proj[..., :C], p["W"], p["bias"], proj[..., C:C + H], p["dt_bias"], p["A_log"],
                                    init=init, output_window=True, cu_seqlens=cu)
    v, k, q = y[..., :H * dv].unflatten(-1, (H, dv)), y[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)), \
        y[..., H * dv + G * dk:].unflatten(-1, (G, dk))
    r = g.ssm_fwd(q, k, v, la, dt, skip=p["skip"], S0=S0, cu_seqlens=cu, save_states=save)
    return r, (y, dt, la, win, q, k, v)


def layer_params(cfg, seed=0):
    H, G, dk, dv = cfg
    gen = torch.Generator().manual_seed(seed)
    C = H * dv + 2 * G * dk
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return {m: t.cuda() for m, t in dict(W=n(C, 4) * 0.5, bias=0.1 * n(C), dt_bias=n(H) - 3, A_log=torch.rand(H, generator=gen) * 2,
                                         skip=n(H)).items()}


@pytest.mark.parametrize("dtype", SCAN)
def test_prompt_then_tokens(dtype):
    """A prompt in two pieces and then single tokens, against the whole at once."""
    import gated_delta_rule_gdn2_b200 as g
    cfg = H, G, dk, dv = 4, 2, 64, 128
    C, T = H * dv + 2 * G * dk, 150
    p = layer_params(cfg)
    proj = torch.randn(2, T, C + H, generator=torch.Generator().manual_seed(5)).to("cuda", TD[dtype])
    (o, ST), _ = layer(g, p, proj, cfg)
    (o1, S), (_, _, _, win, *_) = layer(g, p, proj[:, :70].contiguous(), cfg)
    (o2, S), (_, _, _, win, *_) = layer(g, p, proj[:, 70:140].contiguous(), cfg, init=win, S0=S)
    outs = [o1, o2]
    for t in range(140, T):
        y, dt, la = g.ssm_prologue_step(proj[:, t, :C], p["W"], p["bias"], proj[:, t, C:], p["dt_bias"], p["A_log"], win)
        v, k, q = y[:, :H * dv].unflatten(-1, (H, dv)), y[:, H * dv:H * dv + G * dk].unflatten(-1, (G, dk)), \
            y[:, H * dv + G * dk:].unflatten(-1, (G, dk))
        outs.append(g.ssm_step(q, k, v, la, dt, S, skip=p["skip"])[:, None])
    got = torch.cat(outs, 1).double()
    # each side is within its own bound of the same exact values: 4 operand roundings and 2 results'
    err, ref = (got - o.double()).abs().max().item(), o.double().abs().max().item()
    assert err <= (6 * 2.0 ** -8 if dtype == "bf16" else 1e-5) * ref
    assert (S.double() - ST.double()).norm().item() <= 2e-5 * ST.double().norm().item()
    z = g.output_gate(o, torch.randn_like(o), torch.ones(dv, device="cuda"))
    assert torch.isfinite(z).all() and g.gdn2_get_device_status() == 0


def test_layer_gradients_chain():
    """Prologue and scan differentiated as one layer in fp32, against autograd
    of the fp64 reference, the scan's gradients written straight into the
    prologue's dy."""
    import gated_delta_rule_gdn2_b200 as g
    cfg = H, G, dk, dv = 4, 2, 64, 64
    C = H * dv + 2 * G * dk
    p = layer_params(cfg, 3)
    gen = torch.Generator().manual_seed(6)
    proj = torch.randn(2, 90, C + H, generator=gen).cuda()
    dO = torch.randn(2, 90, H, dv, generator=gen).cuda()
    (o, ST, st), (y, dt, la, _, q, k, v) = layer(g, p, proj, cfg, save=True)
    dy = torch.empty_like(y)
    into = (dy[..., H * dv + G * dk:].unflatten(-1, (G, dk)), dy[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)),
            dy[..., :H * dv].unflatten(-1, (H, dv)))
    gs = g.ssm_bwd(q, k, v, la, dt, dO, skip=p["skip"], states=st, into=into, need_dS0=False)
    gp = g.ssm_prologue_bwd(proj[..., :C], p["W"], p["bias"], proj[..., C:], p["dt_bias"], p["A_log"], dy, gs["ddt"],
                            gs["dlog_alpha"])
    leaf = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    pr = proj.double().cpu().requires_grad_()
    ry, rdt, rla, _ = R.prologue_batch(pr[..., :C], leaf["W"], leaf["bias"], pr[..., C:], leaf["dt_bias"], leaf["A_log"], None)
    ro, _ = R.scan(ry[..., H * dv + G * dk:].unflatten(-1, (G, dk)), ry[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)),
                   ry[..., :H * dv].unflatten(-1, (H, dv)), rla, rdt, leaf["skip"], None)
    want = torch.autograd.grad((ro * dO.double().cpu()).sum(), [pr] + [leaf[n] for n in ("W", "bias", "dt_bias", "A_log", "skip")])
    got = [torch.cat([gp["dx"], gp["dxdt"]], -1), gp["dW"], gp["dbias"], gp["ddt_bias"], gp["dA_log"], gs["dskip"]]
    for a, b in zip(got, want):  # fp32 throughout: a few hundred roundings of 2^-24 in the 2-norm
        assert (host(a) - b).norm() <= 3e-5 * b.norm()


@pytest.mark.parametrize("dtype", SCAN)
def test_captured_and_replayed(dtype):
    """Forward, backward and single tokens in one CUDA graph, replayed on new
    inputs, equal the eager calls bit for bit."""
    import gated_delta_rule_gdn2_b200 as g
    x, y = (make(2, 200, 4, 2, 128, 128, dtype, seed=s) for s in (51, 52))
    d, e = dev(x, dtype), dev(y, dtype)

    def run(d):
        a = [d[n] for n in ("q", "k", "v", "la", "dt")]
        o, ST, st = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True)
        gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st)
        o1 = g.ssm_step(*[t[:, 0].contiguous() for t in a], ST, skip=d["skip"])
        return [o, ST, o1] + [gr[n] for n in GRADS + ("dskip", "dS0")]

    want_d, want_e = run(d), run(e)
    buf = {n: t.clone() for n, t in d.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(buf)
    for src, want in ((d, want_d), (e, want_e), (d, want_d)):
        for n in buf:
            buf[n].copy_(src[n])
        graph.replay()
        for s, t in zip(got, want):
            assert torch.equal(s, t)
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("dtype", SCAN)
def test_two_streams_at_once(dtype):
    """Calls on two streams with workspaces of their own do not touch one another."""
    import gated_delta_rule_gdn2_b200 as g
    d = [dev(make(1, 700, 4, 2, 128, 64, dtype, seed=s), dtype) for s in (61, 62)]

    def run(d, stream=None):
        a = [d[n] for n in ("q", "k", "v", "la", "dt")]
        o, ST, st = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True, stream=stream)
        gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st, stream=stream)
        return [o, ST] + [gr[n] for n in GRADS]

    want = [run(x) for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(3):
        got = []
        for x, s in zip(d, streams):
            with torch.cuda.stream(s):
                got.append(run(x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for s, t in zip(a, b):
                assert torch.equal(s, t)


@pytest.mark.parametrize("dtype", SCAN)
def test_stream_argument_and_rows_before_the_first_sequence(dtype):
    """A stream by its handle while another is current, and offsets that start
    behind row 0: the calls' results, and rows of no sequence as they were."""
    import gated_delta_rule_gdn2_b200 as g
    lens, ahead = (140, 0, 33), 9
    x = make(3, ahead + sum(lens), 4, 2, 64, 64, dtype, lens=(ahead,) + lens, seed=71)
    for n in ("S0", "dS_T"):
        x[n] = x[n][:3]
    d = dev(x, dtype)
    rest = {n: d[n][ahead:].contiguous() for n in ("q", "k", "v", "la", "dt", "dO")}
    cu0 = cu_of(lens)
    cu1 = cu0 + ahead
    names = ("q", "k", "v", "la", "dt")
    W, bias, A, db = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda"), torch.randn(4, device="cuda"), None

    def run(y, cu, **kw):
        a = [y[n] for n in names]
        o, ST, st = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True, cu_seqlens=cu, **kw)
        into = tuple(torch.full_like(t, 5.0) for t in a[:3])
        kw.get("stream") and torch.cuda.current_stream().synchronize()
        gr = g.ssm_bwd(*a, y["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st, cu_seqlens=cu, into=into, **kw)
        xx = y["v"].flatten(1)[:, :64]
        pr = g.ssm_prologue(xx, W, bias, y["dt"], db, A, output_window=True, cu_seqlens=cu, **kw)
        dx = xx.contiguous()
        kw.get("stream") and torch.cuda.current_stream().synchronize()
        gp = g.ssm_prologue_bwd(xx, W, bias, y["dt"], db, A, dx, y["dt"], y["la"], cu_seqlens=cu, **kw)
        return ([o, pr[0], pr[1], pr[2], gp["dx"], gp["dxdt"]] + [gr[n] for n in GRADS],
                [ST, pr[3], gp["dW"], gp["dbias"], gp["dA_log"], gr["dS0"]], into)

    rows, whole, _ = run(rest, cu0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kw in ({}, {"stream": side}, {"stream": side.cuda_stream}):
        r1, w1, into = run(d, cu1, **kw)
        side.synchronize()
        for s, t in zip(rows[:6], r1[:6]):
            assert torch.equal(s, t[ahead:])
        for s, t in zip(whole[:2], w1[:2]):
            assert torch.equal(s, t)
        # (the sums over every token meet other rows in a block, and the packed slots move: fp32 sums in another order)
        for s, t in zip(whole[2:5], w1[2:5]):
            assert (s - t).norm() <= 1e-5 * s.norm()
        for s, t in zip(rows[6:], r1[6:]):
            assert torch.equal(s, t[ahead:])
        assert torch.equal(whole[5], w1[5])
        for t in into:
            assert torch.all(t[:ahead] == 5.0)
    assert g.gdn2_get_device_status() == 0


def test_batches_and_sequences_of_nothing():
    import gated_delta_rule_gdn2_b200 as g
    for B, T in ((0, 5), (2, 0)):
        e = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
        q, v, la, S0 = e(B, T, 1, 64), e(B, T, 2, 64), e(B, T, 2), torch.randn(B, 2, 64, 64, device="cuda")
        o, ST, st = g.ssm_fwd(q, q, v, -la, la, skip=e(2), S0=S0, save_states=True)
        gr = g.ssm_bwd(q, q, v, -la, la, v, skip=e(2), S0=S0, dS_T=2 * S0, states=st)
        assert o.shape == v.shape and torch.equal(ST, S0) and torch.equal(gr["dS0"], 2 * S0)
        assert gr["dq"].shape == q.shape and torch.all(gr["dskip"] == 0)
        x, W, init = e(B, T, 8), e(8, 4), torch.randn(B, 3, 8, device="cuda")
        y, dt, a, win = g.ssm_prologue(x, W, e(8), la, e(2), e(2), init=init, output_window=True)
        assert y.shape == x.shape and torch.equal(win, init) and dt.shape == la.shape
        gp = g.ssm_prologue_bwd(x, W, e(8), la, e(2), e(2), x, la, la, init=init)
        assert torch.all(gp["dW"] == 0) and torch.all(gp["dA_log"] == 0) and torch.all(gp["dinit"] == 0)
    assert g.ssm_step(e(0, 1, 64), e(0, 1, 64), e(0, 2, 64), e(0, 2), e(0, 2), e(0, 2, 64, 64)).shape == (0, 2, 64)
    assert g.gdn2_get_device_status() == 0


def test_arguments_are_checked():
    """What the tensors must be: each of these is refused before anything is launched."""
    import gated_delta_rule_gdn2_b200 as g
    B, T, H, G, dk, dv = 2, 6, 4, 2, 64, 64
    d = dev(make(B, T, H, G, dk, dv, "bf16", seed=81), "bf16")
    d.update(W=torch.randn(dv, 4, device="cuda"), A=torch.randn(H, device="cuda"), cu=cu_of((2, 4)))
    x, win = d["v"][:, :, 0].contiguous(), torch.zeros(B, 3, dv, dtype=torch.bfloat16, device="cuda")

    def fwd(**kw):
        a = {**d, **kw}
        return g.ssm_fwd(*[a[n] for n in ("q", "k", "v", "la", "dt")], skip=a["skip"], S0=a["S0"], cu_seqlens=kw.get("cu"))

    def bwd(**kw):
        a = {**d, **kw}
        return g.ssm_bwd(*[a[n] for n in ("q", "k", "v", "la", "dt", "dO")], skip=a["skip"], S0=a["S0"], dS_T=a["dS_T"],
                         states=kw.get("states"), into=kw.get("into"))

    def step(**kw):
        a = {**{n: t[:, 0].contiguous() for n, t in d.items() if n in ("q", "k", "v", "la", "dt")}, "S": d["S0"].clone(), **kw}
        return g.ssm_step(*[a[n] for n in ("q", "k", "v", "la", "dt", "S")], skip=d["skip"])

    def pro(f=g.ssm_prologue, **kw):
        a = {"x": x, "W": d["W"], "bias": None, "xdt": d["dt"], "dt_bias": None, "A": d["A"], **kw}
        more = {n: a[n] for n in ("init", "cu_seqlens", "ddt", "dlog_alpha") if n in a}
        pos = [a[n] for n in ("dy",) if n in a]
        return f(*[a[n] for n in ("x", "W", "bias", "xdt", "dt_bias", "A")], *pos, **more)

    for f in (fwd, bwd, step, pro):
        if f is not bwd:
            f()
    bad = [
        (fwd, dict(q=d["q"].float())), (fwd, dict(k=d["k"][:, :5])), (fwd, dict(k=d["k"][..., :1, :])),
        (fwd, dict(q=d["q"][:, :, :, ::2], k=d["k"][:, :, :, ::2])), (fwd, dict(v=d["v"].transpose(1, 2))),
        (fwd, dict(la=d["la"].float())), (fwd, dict(la=d["la"].transpose(0, 1))), (fwd, dict(dt=d["dt"][..., :3])),
        (fwd, dict(skip=d["skip"].bfloat16())), (fwd, dict(skip=d["skip"][:2])), (fwd, dict(S0=d["S0"][:1])),
        (fwd, dict(S0=d["S0"].transpose(2, 3))), (fwd, dict(cu=cu_of((2, 4)))), (fwd, dict(q=d["q"].cpu())),
        (fwd, dict(la=d["la"].cpu())), (fwd, dict(v=d["v"][:, :5])), (fwd, dict(v=d["v"][:1].expand(2, -1, -1, -1))),
        (bwd, dict(dO=d["dO"].float())), (bwd, dict(dO=d["dO"][:, :5])), (bwd, dict(dS_T=d["dS_T"].bfloat16())),
        (bwd, dict(states=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
        (bwd, dict(into=(d["q"].float(), d["k"], d["v"]))), (bwd, dict(into=(d["q"], d["k"], d["v"][:, :5]))),
        (step, dict(S=d["S0"].bfloat16())), (step, dict(S=d["S0"][:1])), (step, dict(la=d["la"])),
        (pro, dict(W=d["W"].bfloat16())), (pro, dict(W=d["W"][:8])), (pro, dict(bias=d["A"])), (pro, dict(A=None)),
        (pro, dict(xdt=d["dt"][:, :5])), (pro, dict(xdt=d["dt"].float())), (pro, dict(init=win[:, :2])),
        (pro, dict(x=x.transpose(0, 1))), (pro, dict(dt_bias=d["A"][:2])),
        (pro, dict(f=g.ssm_prologue_bwd, dy=x)), (pro, dict(f=g.ssm_prologue_bwd, dy=x[:, :5], ddt=d["dt"], dlog_alpha=d["dt"])),
    ]
    for i, (f, kw) in enumerate(bad):
        with pytest.raises((ValueError, g.Gdn2Error)):
            f(**kw)
            pytest.fail("case %d (%s) was taken" % (i, list(kw)))
    with pytest.raises(TypeError):
        fwd(q=d["q"].half(), k=d["k"].half(), v=d["v"].half(), la=d["la"].half(), dt=d["dt"].half())
    assert g.gdn2_get_device_status() == 0


@pytest.mark.parametrize("B,H,bad", [(6, 32, False), (64, 4, False), (65, 4, False), (64, 4, True)])
def test_packed_batches_of_many_blocks(B, H, bad):
    """More blocks than SMs, which take the sequences by length: bit for bit
    each sequence alone, equal lengths and empty ones among them, and beside a
    sequence whose offsets are out of range."""
    import gated_delta_rule_gdn2_b200 as g
    lens = [(0, 130, 130, 17, 260, 1, 64)[i % 7] for i in range(B)]
    T = sum(lens)
    d = dev(make(B, T, H, 2, 64, 64, "bf16", lens=lens, seed=91), "bf16")
    names = ("q", "k", "v", "la", "dt")
    cu = cu_of(lens)
    if bad:
        cu[-1] = T + 1
    a = [d[n] for n in names]
    o, ST, st = g.ssm_fwd(*a, skip=d["skip"], S0=d["S0"], save_states=True, cu_seqlens=cu)
    gr = g.ssm_bwd(*a, d["dO"], skip=d["skip"], S0=d["S0"], dS_T=d["dS_T"], states=st, cu_seqlens=cu)
    assert g.gdn2_get_device_status() == (-1 if bad else 0)
    ends = np.cumsum([0] + lens)
    for b in range(B - bad):
        if 14 < b < B - 8:  # (the pattern repeats)
            continue
        s, one = slice(ends[b], ends[b + 1]), slice(b, b + 1)
        x = [t[None, s].contiguous() for t in a]
        ob, Sb = g.ssm_fwd(*x, skip=d["skip"], S0=d["S0"][one])
        gb = g.ssm_bwd(*x, d["dO"][None, s].contiguous(), skip=d["skip"], S0=d["S0"][one], dS_T=d["dS_T"][one])
        for got, want in ((o[s], ob[0]), (ST[b], Sb[0]), (gr["dv"][s], gb["dv"][0]), (gr["dS0"][b], gb["dS0"][0])):
            assert torch.equal(got, want), b
