"""The selective state space scan and its prologue in fp64 torch, token by
token and written from their definitions, with the magnitude sums that error
bounds are taken from.

Bounds.  Every output of the scan is a sum of products, multilinear in q, k,
v, dt, dO, S0, dS_T with non-negative decays as coefficients.  `mag` is that
sum with every factor replaced by its magnitude (the same reference run on
absolute values), so rounding one factor of every product by a relative r
moves the output by at most r mag.
  fp32: n roundings of 2^-24 along a sum (n below), 2^-20 for the fast
  exponential: |err| <= (n 2^-24 + 2^-20) mag.
  bf16 outputs: one rounding of the result, 2^-8 |ref|, and the operands that
  the tensor cores take in bf16: at most `ops` of them in a product.
  fp32 outputs of bf16 inputs (states, dskip): operands in two bf16 parts,
  2^-16 mag.
"""
import numpy as np
import torch

F64 = torch.float64


def scan(q, k, v, la, dt, skip, S0, lens=None):
    """o, S_T (fp64).  [B, T, ..], or packed [rows, ..] with lens; rows past
    the last sequence stay zero."""
    if lens is not None:
        o, S, r = torch.zeros_like(v), [], 0
        parts = []
        for b, n in enumerate(lens):
            x = [t[None, r:r + n] for t in (q, k, v, la, dt)]
            ob, Sb = scan(*x, skip, None if S0 is None else S0[b:b + 1])
            parts.append(ob[0])
            S.append(Sb)
            r += n
        o = torch.cat(parts + [torch.zeros_like(v[r:])])
        return o, torch.cat(S)
    B, T, H, dv = v.shape
    r, dk = H // q.shape[2], q.shape[3]
    S = torch.zeros(B, H, dk, dv, dtype=v.dtype) if S0 is None else S0
    outs = []
    for t in range(T):
        kt, qt = (x[:, t].repeat_interleave(r, 1) for x in (k, q))
        S = la[:, t].exp()[..., None, None] * S + (dt[:, t, :, None] * kt)[..., None] * v[:, t, :, None, :]
        o = (qt[..., None] * S).sum(-2)
        outs.append(o if skip is None else o + skip[:, None] * v[:, t])
    return (torch.stack(outs, 1) if T else v.clone()), S


def scan_grads(q, k, v, la, dt, skip, S0, dO, dS_T, lens=None):
    """o, S_T and the gradients of every input given."""
    x = [None if t is None else t.clone().requires_grad_() for t in (q, k, v, la, dt, skip, S0)]
    o, ST = scan(*x, lens=lens)
    loss = (o * dO).sum() + (0 if dS_T is None else (ST * dS_T).sum())
    have = [t for t in x if t is not None]
    g = iter(torch.autograd.grad(loss, have, allow_unused=True, materialize_grads=True))
    names = ("dq", "dk", "dv", "dlog_alpha", "ddt", "dskip", "dS0")
    out = {"o": o.detach(), "S_T": ST.detach()}
    out.update({n: None if t is None else next(g) for n, t in zip(names, x)})
    return out


def magnitudes(q, k, v, la, dt, skip, S0, dO, dS_T, lens=None):
    """mag of every output; for dlog_alpha with the rounding of its running
    sum, as a bound to add ("dla_sum").

    dlog_alpha_t holds sum_{i >= t > j} W_ij over a chunk of at most 128
    tokens, taken as the sum over i >= t of (row sum - column sum) of the W_ij
    below the diagonal.  Each sum has at most 127 terms and the running sum 128
    more, in trees or runs of at most 64 + 16 roundings, each of at most 2^-24
    of what is summed.  All of it is at most the sum over the chunk of
    |do_i| . mag o_i (the rows) and dt_j mag ddt_j (the columns), here taken
    over 128 tokens either way: 80 2^-24 < 2^-17 of that sum."""
    ab = lambda t: None if t is None else t.abs()  # noqa: E731
    m = scan_grads(ab(q), ab(k), ab(v), la, dt, ab(skip), ab(S0), ab(dO), ab(dS_T), lens)
    row = ab(dO) * (m["o"] if skip is None else m["o"] - skip.abs()[:, None] * v.abs())
    near = row.sum(-1) + dt * m["ddt"]
    near = near.unsqueeze(0) if lens is not None else near  # [B, T, H]
    c = torch.nn.functional.pad(near.cumsum(1), (0, 0, 1, 0))
    T = near.shape[1]
    at = torch.arange(T)
    near = c[:, (at + 129).clamp(max=T)] - c[:, (at - 128).clamp(min=0)]
    m["dla_sum"] = 2.0 ** -17 * (near[0] if lens is not None else near)
    return m


def prologue(x, W, bias, xdt, dt_bias, A_log, init):
    """y, dt, la, window of one sequence [T, C]."""
    K, T = W.shape[1], x.shape[0]
    w = torch.cat([torch.zeros(K - 1, x.shape[1], dtype=F64) if init is None else init, x])
    u = torch.zeros_like(x) if bias is None else bias.expand_as(x)
    for j in range(K):
        u = u + W[:, j] * w[j:j + T]
    dt = la = None
    if xdt is not None:
        z = xdt if dt_bias is None else xdt + dt_bias
        dt = torch.logaddexp(z, torch.zeros_like(z))
        la = -A_log.exp() * dt
    return u / (1 + torch.exp(-u)), dt, la, w[T:]


def prologue_batch(x, W, bias, xdt, dt_bias, A_log, init, lens=None):
    """Of a batch [B, T, ..] or packed rows."""
    seqs = list(range(x.shape[0])) if lens is None else \
        [slice(a, a + n) for a, n in zip(np.cumsum([0] + list(lens[:-1])), lens)]
    r = [prologue(x[s], W, bias, None if xdt is None else xdt[s], dt_bias, A_log, None if init is None else init[b])
         for b, s in enumerate(seqs)]
    join = torch.stack if lens is None else torch.cat
    return [None if r[0][i] is None else join([t[i] for t in r]) for i in range(3)] + [torch.stack([t[3] for t in r])]


def sums_bound(T, dk, dv):
    """Relative bound of a fp32 sum along T tokens of a dk x dv state."""
    return (2 * T + dk + dv + 64) * 2.0 ** -24 + 2.0 ** -20


def within(name, x, ref, mag, rel, out_rel=0.0, more=0.0):
    """|x - ref| <= rel mag + out_rel |ref| + more, entry by entry."""
    x, ref, mag = (np.asarray(t, np.float64) for t in (x, ref, mag))
    assert x.shape == ref.shape, (name, x.shape, ref.shape)
    assert np.all(np.isfinite(x)), "%s: not finite" % name
    over = np.abs(x - ref) - (rel * mag + out_rel * np.abs(ref) + np.asarray(more) + 1e-30)
    worst = float(over.max()) if over.size else 0.0
    if worst > 0:
        at = np.unravel_index(int(over.argmax()), over.shape)
        raise AssertionError("%s%s: %g, want %g, off by %g, allowed %g" % (
            name, tuple(int(i) for i in at), x[at], ref[at], abs(x[at] - ref[at]), abs(x[at] - ref[at]) - worst))
