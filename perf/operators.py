"""The selective state space operators as a user's program calls them, beside
their plain forms.

A scan over T tokens with heads h and groups g(h) = h // (H / G):

    S_t = e^{la_t} S_{t-1} + dt_t k_t v_t^T        (S: dk x dv, fp32)
    o_t = S_t^T q_t + skip_h v_t

(q = C, k = B and v = x in the usual names of a state space layer), and the
layer's prologue: y = silu(conv(x) + bias), a depthwise causal convolution over
K taps that starts from the K - 1 inputs before the first one, with
dt = softplus(xdt + dt_bias) and la = -exp(A_log) dt.

`own` is false for the plain forms and true for the package's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# ---------------------------------------------------------------------------
# cases.  Sizes: 16 heads of 128 channels and a 128-channel state, batches of
# 8 x 4096 tokens, decoding batches of 256 and long sequences of 32768 tokens
# are the package's own workloads; C channels of a prologue = H dv + 2 G dk.


def _scan(kind, B, T, H, G, dk, dv, dtype="bf16", packed=False, strided=False, s0=True):
    return {"kind": kind, "B": B, "T": T, "H": H, "G": G, "dk": dk, "dv": dv, "dtype": dtype, "packed": packed,
            "strided": strided, "s0": s0}


def _conv(kind, B, T, H, C, K, dtype="bf16", packed=False, init=False):
    return {"kind": kind, "B": B, "T": T, "H": H, "C": C, "K": K, "dtype": dtype, "packed": packed, "init": init}


def listed():
    return [
        # one sequence being answered: the latency of a single token
        {"name": "step B1", **_scan("step", 1, 1, 16, 1, 128, 128)},
        # a full decoding batch
        {"name": "step B256", **_scan("step", 256, 1, 16, 1, 128, 128)},
        # a short prompt that continues a cached one, of odd length
        {"name": "prompt B1 T200", **_scan("prompt", 1, 200, 16, 1, 128, 128)},
        # a batch of prompts
        {"name": "prompt B8 T4096", **_scan("prompt", 8, 4096, 16, 1, 128, 128)},
        # a long document, q, k, v as views of the convolution's output
        {"name": "prompt B1 T32768 strided", **_scan("prompt", 1, 32768, 16, 1, 128, 128, strided=True, s0=False)},
        # packed prompts of different lengths, smaller heads in two groups
        {"name": "prompt packed 12 x 9001", **_scan("prompt", 12, 9001, 32, 2, 128, 64, packed=True)},
        # a training step
        {"name": "train B8 T4096", **_scan("train", 8, 4096, 16, 1, 128, 128, s0=False)},
        # training in fp32 on small heads
        {"name": "train fp32 B2 T1000", **_scan("train", 2, 1000, 8, 2, 64, 64, dtype="fp32")},
        # the convolution's single token
        {"name": "conv step B256", **_conv("conv step", 256, 1, 16, 2304, 4)},
        # a batch of prompts, each continuing its cached window
        {"name": "conv prompt B8 T4096", **_conv("conv prompt", 8, 4096, 16, 2304, 4, init=True)},
        # a training step on packed documents
        {"name": "conv train packed 9 x 16387", **_conv("conv train", 9, 16387, 16, 2304, 4, packed=True)},
        # training in fp32, an odd length
        {"name": "conv train fp32 B3 T777", **_conv("conv train", 3, 777, 8, 640, 3, dtype="fp32", init=True)},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["step", "prompt", "prompt", "train", "train", "conv step", "conv prompt", "conv train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    G = rng.choice([1, 1, 2, 4])
    H = G * rng.choice([1, 2, 4, 8] if G > 1 else [1, 3, 8, 16])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
    packed = rng.random() < 0.4
    if kind in ("step", "conv step"):
        B = log_int(1, 256)
        if kind == "conv step":
            return _conv(kind, B, 1, H, H * dv + 2 * G * dk, rng.randint(2, 4), dtype, init=True)
        return _scan(kind, B, 1, H, G, dk, dv, dtype, strided=rng.random() < 0.5)
    rows = log_int(1, 24000 if dtype == "bf16" else 6000)  # all the tokens of the call
    if kind == "train":
        rows = max(2, rows // 2)
    B = log_int(1, min(rows, 16))
    T = rows if packed else max(1, rows // B)
    if kind.startswith("conv"):
        return _conv(kind, B, T, H, H * dv + 2 * G * dk, rng.randint(1, 4), dtype, packed, rng.random() < 0.5)
    return _scan(kind, B, T, H, G, dk, dv, dtype, packed, rng.random() < 0.5, rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs


def _lengths(B, T, seed):
    """B lengths that sum to T: of any size, among them an empty one where B > 2."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, T + 1, (B - 1,), generator=g)).values.tolist()
    if B > 2:
        cuts[1] = cuts[0]
    e = [0] + cuts + [T]
    return [e[i + 1] - e[i] for i in range(B)]


def prepare(case, seed):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    B, T, H = case["B"], case["T"], case["H"]
    st = {"case": case, "lens": None, "cu": None}
    if case["packed"]:
        st["lens"] = _lengths(B, T, seed)
        offs = [0]
        for x in st["lens"]:
            offs.append(offs[-1] + x)
        st["cu"] = torch.tensor(offs, dtype=torch.int32, device=dev)
    lead = (B,) if "step" in case["kind"] else (T,) if case["packed"] else (B, T)
    # A in 1 .. 16 and steps dt of 0.001 .. 0.1, as such a layer is initialised
    A_log = torch.log(torch.rand(H, generator=gen, device=dev) * 15 + 1)
    dt0 = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(100) + math.log(1e-3))
    dt_bias = dt0 + torch.log(-torch.expm1(-dt0))  # softplus(dt_bias) = dt0
    if "conv" in case["kind"]:
        C, K = case["C"], case["K"]
        # the projection's output: [gate | channels | step], read in place
        proj = n(*lead, 64 + C + H).to(dt)
        st.update(x=proj[..., 64:64 + C], xdt=proj[..., 64 + C:], W=n(C, K) * K ** -0.5, bias=0.1 * n(C),
                  A_log=A_log, dt_bias=dt_bias)
        st["init"] = n(B, K - 1, C).to(dt) if case["init"] or "step" in case["kind"] else None
        if case["kind"] == "conv train":
            st.update(dy=n(*lead, C).to(dt), ddt=n(*lead, H).to(dt), dla=n(*lead, H).to(dt))
        return st
    G, dk, dv = case["G"], case["dk"], case["dv"]
    # the convolution's output is a SiLU of values of order one
    xBC = torch.nn.functional.silu(n(*lead, H * dv + 2 * G * dk)).to(dt)
    v, k, q = torch.split(xBC, [H * dv, G * dk, G * dk], dim=-1)
    v, k, q = v.unflatten(-1, (H, dv)), k.unflatten(-1, (G, dk)), q.unflatten(-1, (G, dk))
    if not case["strided"]:
        v, k, q = v.contiguous(), k.contiguous(), q.contiguous()
    step = torch.nn.functional.softplus(n(*lead, H) + dt_bias)
    st.update(q=q, k=k, v=v, dt=step.to(dt), la=(-torch.exp(A_log) * step).to(dt), skip=1 + 0.1 * n(H))
    st["S0"] = 0.1 * n(B, H, dk, dv) if case["s0"] or case["kind"] == "step" else None
    if case["kind"] == "train":
        st["dO"] = n(*lead, H, dv).to(dt)
        st["dST"] = 0.1 * n(B, H, dk, dv) if case["s0"] else None
    return st


# ---------------------------------------------------------------------------
# plain forms, in 32 bits (log decays summed in 64)


def _pad_rows(x, lens, Tmax):
    """[rows, ...] of packed sequences -> [B, Tmax, ...], zeros behind each."""
    return torch.nn.utils.rnn.pad_sequence(list(torch.split(x, lens)), batch_first=True) if Tmax else x[None]


def _unpad_rows(x, lens):
    keep = torch.arange(x.shape[1], device=x.device)[None] < torch.tensor(lens, device=x.device)[:, None]
    return x[keep]


def _plain_scan(q, k, v, la, dt, skip, S0):
    """o, S_T of [B, T, ...] fp32 tensors: chunks of 64 tokens, the states at
    their borders from the decays between chunks."""
    B, T, H, dv = v.shape
    G, dk = q.shape[2], q.shape[3]
    C = 64
    n = -(-T // C)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * C - T))  # noqa: E731
    q, k = (pad(x).reshape(B, n, C, G, 1, dk).expand(B, n, C, G, H // G, dk).reshape(B, n, C, H, dk) for x in (q, k))
    vp, dtp = pad(v).reshape(B, n, C, H, dv), pad(dt).reshape(B, n, C, H)
    L = pad(la.double()).reshape(B, n, C, H).cumsum(2)  # decay since the chunk's start
    end = L[:, :, -1]
    tri = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    W = (L[:, :, :, None] - L[:, :, None]).masked_fill(~tri[None, None, :, :, None], -torch.inf).exp().float()
    M = torch.einsum("bnihd,bnjhd->bnijh", q, k) * W * dtp[:, :, None]
    o = torch.einsum("bnijh,bnjhp->bnihp", M, vp)
    # each chunk's own contribution to the state at its end
    wk = (end[:, :, None] - L).exp().float() * dtp
    own_S = torch.einsum("bnjhd,bnjhp->bnhdp", k * wk[..., None], vp)
    # states at chunk starts (and after the last): the contributions before, decayed
    tot = torch.cat([torch.zeros_like(end[:, :1]), end.cumsum(1)], 1)  # [B, n + 1, H]
    at, of = torch.arange(n + 1, device=v.device)[:, None], torch.arange(n, device=v.device)[None]
    D = (tot[:, :, None] - tot[:, None, 1:]).masked_fill(~(of < at)[None, :, :, None], -torch.inf).exp().float()
    S = torch.einsum("bmnh,bnhdp->bmhdp", D, own_S)
    if S0 is not None:
        S = S + tot.exp().float()[..., None, None] * S0[:, None]
    o = o + torch.einsum("bnihd,bnhdp->bnihp", q * L.exp().float()[..., None], S[:, :-1])
    o = o.reshape(B, n * C, H, dv)[:, :T] + skip[:, None] * v
    return o, S[:, -1]


def _plain_conv(x, xdt, W, bias, A_log, dt_bias, init):
    """y, dt, la and the window after the last token, of [B, T, ...] fp32."""
    K, T = W.shape[1], x.shape[1]
    w = torch.cat([x.new_zeros(x.shape[0], K - 1, x.shape[2]) if init is None else init, x], 1)
    u = (w.unfold(1, K, 1)[:, :T] * W).sum(-1) + bias
    dt = torch.nn.functional.softplus(xdt + dt_bias, threshold=40.0)
    return u * torch.sigmoid(u), dt, -torch.exp(A_log) * dt, w[:, T:]


def _batch(st, names):
    """The named inputs in 32 bits, as [B, T, ...]."""
    lens, f = st["lens"], [st[m].float() for m in names]
    return f if lens is None else [_pad_rows(x, lens, max(lens)) for x in f]


def _window_after(x, init, lens, K):
    """Packed: each sequence's last K - 1 inputs, its initial window before them."""
    B, C = len(lens), x.shape[-1]
    z = x.new_zeros(B, K - 1, C) if init is None else init
    at = torch.tensor(lens, device=x.device)[:, None] + torch.arange(K - 1, device=x.device)[None]
    full = torch.cat([z, _pad_rows(x, lens, max(lens))], 1)
    return torch.gather(full, 1, at[..., None].expand(B, K - 1, C))


def _run_plain(st):
    case = st["case"]
    kind, lens, dtype = case["kind"], st["lens"], DTYPES[case["dtype"]]
    flat = (lambda x: x) if lens is None else (lambda x: _unpad_rows(x, lens))
    if kind == "step":
        H, G = case["H"], case["G"]
        q, k = (st[m].float().repeat_interleave(H // G, 1) for m in ("q", "k"))
        v, dt, a = st["v"].float(), st["dt"].float(), st["la"].float().exp()
        S = st["S0"].mul_(a[..., None, None]).add_((dt[..., None] * k)[..., None] * v[..., None, :])  # kept in place
        return (torch.einsum("bhd,bhdp->bhp", q, S) + st["skip"][:, None] * v).to(dtype), S
    if kind == "prompt":
        o, ST = _plain_scan(*_batch(st, ("q", "k", "v", "la", "dt")), st["skip"], st["S0"])
        return flat(o).to(dtype), ST
    if kind == "train":
        x = [t.requires_grad_() for t in _batch(st, ("q", "k", "v", "la", "dt"))]
        skip = st["skip"].clone().requires_grad_()
        S0 = None if st["S0"] is None else st["S0"].clone().requires_grad_()
        o, ST = _plain_scan(*x, skip, S0)
        outs, ups = [o], _batch(st, ("dO",))
        if st["dST"] is not None:
            outs, ups = [o, ST], ups + [st["dST"]]
        g = torch.autograd.grad(outs, x + [skip] + ([] if S0 is None else [S0]), ups)
        return [flat(o.detach()).to(dtype), ST.detach(), [flat(t).to(dtype) for t in g[:5]], list(g[5:])]
    if kind == "conv step":
        x, xdt = st["x"].float()[:, None], st["xdt"].float()[:, None]
        y, dt, la, win = _plain_conv(x, xdt, st["W"], st["bias"], st["A_log"], st["dt_bias"], st["init"].float())
        return y[:, 0].to(dtype), dt[:, 0].to(dtype), la[:, 0].to(dtype), st["init"].copy_(win)  # kept in place
    init = None if st["init"] is None else st["init"].float()
    x, xdt = _batch(st, ("x", "xdt"))
    if kind == "conv prompt":
        y, dt, la, win = _plain_conv(x, xdt, st["W"], st["bias"], st["A_log"], st["dt_bias"], init)
        if lens is not None:
            win = _window_after(st["x"].float(), init, lens, case["K"])
        return flat(y).to(dtype), flat(dt).to(dtype), flat(la).to(dtype), win.to(dtype)
    w = [t.clone().requires_grad_() for t in (st["W"], st["bias"], st["A_log"], st["dt_bias"])]
    x, xdt = x.requires_grad_(), xdt.requires_grad_()
    init = None if init is None or case["K"] == 1 else init.requires_grad_()
    y, dt, la, _ = _plain_conv(x, xdt, *w, init)
    if lens is not None:  # nothing comes back from behind a sequence's end
        keep = (torch.arange(x.shape[1], device=x.device)[None] < torch.tensor(lens, device=x.device)[:, None])[..., None]
        y, dt, la = y * keep, dt * keep, la * keep
    g = torch.autograd.grad([y, dt, la], [x, xdt] + w + ([] if init is None else [init]), _batch(st, ("dy", "ddt", "dla")))
    return [flat(t.detach()).to(dtype) for t in (y, dt, la)] + [flat(t).to(dtype) for t in g[:2]] + list(g[2:6]) + \
        [t.to(dtype) for t in g[6:]]


# ---------------------------------------------------------------------------
# the package's operators


def _run_own(st):
    import gated_delta_rule_gdn2_b200 as g
    case = st["case"]
    kind, cu = case["kind"], st["cu"]
    if kind == "step":
        return g.ssm_step(st["q"], st["k"], st["v"], st["la"], st["dt"], st["S0"], skip=st["skip"]), st["S0"]
    if kind == "prompt":
        return g.ssm_fwd(st["q"], st["k"], st["v"], st["la"], st["dt"], skip=st["skip"], S0=st["S0"], cu_seqlens=cu)
    if kind == "train":
        x = (st["q"], st["k"], st["v"], st["la"], st["dt"])
        o, ST, states = g.ssm_fwd(*x, skip=st["skip"], S0=st["S0"], save_states=True, cu_seqlens=cu)
        r = g.ssm_bwd(*x, st["dO"], skip=st["skip"], S0=st["S0"], dS_T=st["dST"], states=states,
                      need_dS0=st["S0"] is not None, cu_seqlens=cu)
        rest = [r["dskip"]] + ([] if st["S0"] is None else [r["dS0"]])
        return [o, ST, [r[m] for m in ("dq", "dk", "dv", "dlog_alpha", "ddt")], rest]
    w = (st["W"], st["bias"], st["xdt"], st["dt_bias"], st["A_log"])
    if kind == "conv step":
        y, dt, la = g.ssm_prologue_step(st["x"], *w, st["init"])
        return y, dt, la, st["init"]
    if kind == "conv prompt":
        return g.ssm_prologue(st["x"], *w, init=st["init"], output_window=True, cu_seqlens=cu)
    y, dt, la, _ = g.ssm_prologue(st["x"], *w, init=st["init"], cu_seqlens=cu)
    r = g.ssm_prologue_bwd(st["x"], *w, st["dy"], st["ddt"], st["dla"], init=st["init"], cu_seqlens=cu)
    rest = [] if st["init"] is None or case["K"] == 1 else [r["dinit"]]
    return [y, dt, la] + [r[m] for m in ("dx", "dxdt", "dW", "dbias", "dA_log", "ddt_bias")] + rest


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T, H, kind = case["B"], case["T"], case["H"], case["kind"]
    rows = T if case["packed"] else B * T
    if "conv" in kind:
        C, K = case["C"], case["K"]
        par = 4 * (C * (K + 1) + 2 * H)
        win = B * (K - 1) * C * e
        fwd = rows * (2 * C + 3 * H) * e + par
        if kind == "conv step":
            return {"bytes": fwd + 2 * win, "flops": rows * C * (2 * K + 5)}
        if kind == "conv prompt":
            return {"bytes": fwd + (2 if case["init"] else 1) * win, "flops": rows * C * (2 * K + 5)}
        # forward outputs, then x, dy in and dx out, with the filters' gradients
        return {"bytes": rows * (4 * C + 6 * H) * e + 2 * par + (2 * win if case["init"] else 0),
                "flops": rows * C * (6 * K + 15)}
    G, dk, dv = case["G"], case["dk"], case["dv"]
    inp = rows * (H * dv + 2 * G * dk + 2 * H) * e
    S = 4 * B * H * dk * dv
    if kind == "step":
        return {"bytes": inp + rows * H * dv * e + 2 * S + 4 * H, "flops": 5 * rows * H * dk * dv}
    if kind == "prompt":
        return {"bytes": inp + rows * H * dv * e + (2 if case["s0"] else 1) * S + 4 * H, "flops": 4 * rows * H * dk * dv}
    # o and S_T, do (and dS_T) in, a gradient for each input
    return {"bytes": 2 * inp + 2 * rows * H * dv * e + (4 if case["s0"] else 1) * S + 8 * H,
            "flops": 14 * rows * H * dk * dv}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token


def _exact_scan(q, k, v, la, dt, skip, S, dO=None, dS=None):
    """One batch [B, T, ...] of equal lengths: o and S_T, and with dO the gradients too."""
    B, T, H, dv = v.shape
    r = H // q.shape[2]
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    a = la.exp()
    o, starts = torch.empty_like(v), []
    every = 32

    def forward(S, t):
        return a[:, t, :, None, None] * S + torch.einsum("bhd,bhp->bhdp", k[:, t] * dt[:, t, :, None], v[:, t])

    for t in range(T):
        if dO is not None and t % every == 0:
            starts.append(S)
        S = forward(S, t)
        o[:, t] = torch.einsum("bhd,bhdp->bhp", q[:, t], S) + skip[:, None] * v[:, t]
    ST = S
    if dO is None:
        return o, ST
    dq, dk, dv_, dla, ddt = (torch.empty_like(x) for x in (q, k, v, la, dt))
    for c in range(len(starts) - 1, -1, -1):
        lo, hi = c * every, min(T, (c + 1) * every)
        before = [starts[c]]
        for t in range(lo, hi):
            before.append(forward(before[-1], t))
        starts[c] = None
        for t in range(hi - 1, lo - 1, -1):
            S0, S1 = before[t - lo], before[t - lo + 1]
            dS = dS + torch.einsum("bhd,bhp->bhdp", q[:, t], dO[:, t])
            dq[:, t] = torch.einsum("bhdp,bhp->bhd", S1, dO[:, t])
            kS = torch.einsum("bhdp,bhd->bhp", dS, k[:, t])
            dv_[:, t] = dt[:, t, :, None] * kS + skip[:, None] * dO[:, t]
            ddt[:, t] = (kS * v[:, t]).sum(-1)
            dk[:, t] = dt[:, t, :, None] * torch.einsum("bhdp,bhp->bhd", dS, v[:, t])
            dla[:, t] = a[:, t] * torch.einsum("bhdp,bhdp->bh", dS, S0)
            dS = a[:, t, :, None, None] * dS
    sum_g = lambda x: x.unflatten(2, (H // r, r)).sum(3)  # noqa: E731
    return o, ST, sum_g(dq), sum_g(dk), dv_, dla, ddt, (dO * v).sum((0, 1, 3)), dS


def _exact_conv(x, xdt, W, bias, A_log, dt_bias, win, up=None):
    """One sequence [T, ...]: y, dt, la, the window after it; with up = (dy, ddt, dla) the gradients."""
    K, T = W.shape[1], x.shape[0]
    w = torch.cat([win, x])
    u = bias.expand(T, -1).clone()
    for j in range(K):
        u = u + W[:, j] * w[j:j + T]
    s = 1 / (1 + torch.exp(-u))
    z = xdt + dt_bias
    dt = torch.logaddexp(z, torch.zeros_like(z))
    A = -torch.exp(A_log)
    if up is None:
        return u * s, dt, A * dt, w[T:]
    dy, ddt, dla = up
    du = dy * s * (1 + u * (1 - s))
    dw, dW = torch.zeros_like(w), torch.zeros_like(W)
    for j in range(K):
        dw[j:j + T] += W[:, j] * du
        dW[:, j] = (du * w[j:j + T]).sum(0)
    dz = (ddt + A * dla) / (1 + torch.exp(-z))
    return u * s, dt, A * dt, dw[K - 1:], dz, dW, du.sum(0), (A * dla * dt).sum(0), dz.sum(0), dw[:K - 1]


def exact(case, seed):
    st = prepare(case, seed)
    d = lambda m: None if st[m] is None else st[m].double()  # noqa: E731
    kind, B = case["kind"], case["B"]
    if case["packed"]:
        edges = [0]
        for x in st["lens"]:
            edges.append(edges[-1] + x)
        parts = [slice(edges[i], edges[i + 1]) for i in range(B)]
    if "conv" in kind:
        C, K = case["C"], case["K"]
        wts = [d(m) for m in ("W", "bias", "A_log", "dt_bias")]
        z = d("init") if st["init"] is not None else torch.zeros(B, K - 1, C, dtype=torch.float64, device="cuda")
        x, xdt = d("x"), d("xdt")
        if kind == "conv step":
            r = [_exact_conv(x[b:b + 1], xdt[b:b + 1], *wts, z[b]) for b in range(B)]
            return [torch.cat([t[i] for t in r]) for i in range(3)] + [torch.stack([t[3] for t in r])]
        seqs = parts if case["packed"] else list(range(B))
        if kind == "conv prompt":
            r = [_exact_conv(x[s], xdt[s], *wts, z[b]) for b, s in enumerate(seqs)]
            join = torch.cat if case["packed"] else torch.stack
            return [join([t[i] for t in r]) for i in range(3)] + [torch.stack([t[3] for t in r])]
        ups = [d(m) for m in ("dy", "ddt", "dla")]
        r = [_exact_conv(x[s], xdt[s], *wts, z[b], [u[s] for u in ups]) for b, s in enumerate(seqs)]
        join = torch.cat if case["packed"] else torch.stack
        out = [join([t[i] for t in r]) for i in range(5)] + [sum(t[i] for t in r) for i in range(5, 9)]
        return out + ([] if st["init"] is None or K == 1 else [torch.stack([t[9] for t in r])])
    H, dk, dv = case["H"], case["dk"], case["dv"]
    S = d("S0") if st["S0"] is not None else torch.zeros(B, H, dk, dv, dtype=torch.float64, device="cuda")
    x, skip = [d(m) for m in ("q", "k", "v", "la", "dt")], d("skip")
    if kind == "step":
        o, ST = _exact_scan(*[t[:, None] for t in x], skip, S)
        return o[:, 0], ST
    up = [None, None]
    if kind == "train":
        up = [d("dO"), d("dST") if st["dST"] is not None else torch.zeros_like(S)]
    if not case["packed"]:
        r = _exact_scan(*x, skip, S, *up)
    else:
        each = []
        for b, s in enumerate(parts):
            u = [None, None] if up[0] is None else [up[0][None, s], up[1][b:b + 1]]
            each.append(_exact_scan(*[t[None, s] for t in x], skip, S[b:b + 1], *u))
        cat = lambda i: torch.cat([t[i][0] for t in each])  # noqa: E731
        r = [cat(0), torch.cat([t[1] for t in each])]
        if up[0] is not None:
            r += [cat(i) for i in range(2, 7)] + [sum(t[7] for t in each), torch.cat([t[8] for t in each])]
    if kind == "prompt":
        return r[0], r[1]
    return [r[0], r[1], list(r[2:7]), [r[7]] + ([] if st["S0"] is None else [r[8]])]
