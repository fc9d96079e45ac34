"""Gradients compared in the 2-norm, head by head.

The entry-wise bounds of ssm_ref.py hold for any signs of what is summed, so
they are as large as the sum of the terms' magnitudes: for dlog_alpha and ddt,
inner products of random signs, that is as large as the gradient itself.  On
inputs of independent signs the norm of a whole gradient tells far more.

A rounding to bf16 moves one factor of a product by a relative r, |r| <= 2^-8,
of either sign alike, rms at most 2^-8 / sqrt(3).  Terms of independent signs
are orthogonal on average, so the rounding of one factor moves the gradient by
that rms relative to its own norm, and `ops` such factors and the rounding of
the result by sqrt(ops + 1) / sqrt(3) 2^-8: 1.2 2^-8 for the three of a
gradient.  A few hundred entries a head make the norms themselves uncertain by a
tenth; 4 2^-8 leaves a factor of three over both, and is a third of what a
gradient that is a twentieth too large would show.
  fp32 outputs of bf16 inputs (operands in two bf16 parts): 2^-16 in their place.
  fp32: sums of at most 512 terms, each rounding 2^-24 of the partial sum and
of independent signs: sqrt(512) 2^-24 < 2^-19; 2^-16 leaves a factor of eight
for the products' own roundings and the exponentials.
"""
import torch

BF16, PARTS, FP32 = 4 * 2.0 ** -8, 4 * 2.0 ** -16, 2.0 ** -16


def worst(x, ref, head):
    """The largest |x - ref|_2 / |ref|_2 over the slices along axis `head`."""
    x, ref = (t.to(torch.float64).movedim(head, 0).flatten(1) for t in (x, ref))
    err, size = (x - ref).norm(dim=1), ref.norm(dim=1)
    assert bool(torch.isfinite(x).all()) and bool((size > 0).all())
    return float((err / size).max())


def close(name, x, ref, rel, head):
    w = worst(x, ref, head)
    assert w <= rel, "%s: a head is off by %.3g of its norm, allowed %.3g" % (name, w, rel)
    return w
