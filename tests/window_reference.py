"""Windowed attention in 64 bits, from its definition, for the tests.

A query at position p sees key j <= p when j > p - window or j < sinks.
Besides each result, the functions return how far a kernel's may be off:

* a rounding to bf16 is off by at most U = 2^-8 of the value;
* the kernels round the softmax weights P to bf16 and normalise with the sum
  of the rounded ones, so O = sum P v / sum P is off by at most
  U (sum P |v| + |O|), and by U |O| for its own rounding;
* they round P and dS = P (dP - D) to bf16, and D = rowsum(dO O) is formed
  from O as rounded above, U_O off: dS is off by at most
  P (2 U |dP - D| + sum |dO| U_O), and the products follow linearly;
* fp32 sums and the base-2 exponential add at most 2^-17 of the sums of
  magnitudes here (a few hundred terms of 2^-24 each, and 2^-22).
"""

from __future__ import annotations

import math

U = 2.0 ** -8    # half a step of bf16, relative
F = 2.0 ** -17   # fp32 sums and exponentials, relative to the sums of magnitudes
LSE_TOL = 1e-3   # scores of a few units in fp32, sums of a few thousand terms


def visible(n_q, n_k, first, window, sinks, device):
    """[n_q, n_k] mask; the first query stands at position `first`."""
    import torch
    p = first + torch.arange(n_q, device=device)[:, None]
    j = torch.arange(n_k, device=device)
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def forward(q, k, v, window, sinks, first=None, scale=None):
    """Rows q [n, d] over keys [L, d], float64; the queries are the last n
    positions unless `first` says where they start.  Returns (out, lse,
    tolerance of out)."""
    import torch
    n, d = q.shape
    L = k.shape[0]
    first = L - n if first is None else first
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    x = (q @ k.T) * scale
    x = x.masked_fill(~visible(n, L, first, window, sinks, q.device), -math.inf)
    lse = torch.logsumexp(x, 1) if L else torch.full((n,), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.where(lse[:, None] == -math.inf, 0.0, torch.exp(x - lse[:, None]))
    out = p @ v
    size = p @ v.abs()
    return out, lse, U * (size + 2 * out.abs()) * 1.05 + F * size + 1e-30


def backward(q, k, v, dout, window, sinks, scale=None):
    """Gradients of one head's rows (self-attention) and their tolerances:
    ((dq, dk, dv), (tq, tk, tv))."""
    import torch
    n, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    x = (q @ k.T) * scale
    x = x.masked_fill(~visible(n, n, 0, window, sinks, q.device), -math.inf)
    p = torch.softmax(x, 1)
    out = p @ v
    t_out = U * (p @ v.abs() + 2 * out.abs())
    dp = dout @ v.T
    D = (dout * out).sum(1, keepdim=True)
    e = dp - D
    ds = p * e
    t_ds = p * (2 * U * e.abs() + (dout.abs() * t_out).sum(1, keepdim=True)
                + F * ((dout.abs() @ v.abs().T) + (dout * out).abs().sum(1, keepdim=True)))
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ dout
    tq = scale * (t_ds + F * ds.abs()) @ k.abs()
    tk = scale * (t_ds + F * ds.abs()).T @ q.abs()
    tv = (U + F) * p.T @ dout.abs()
    return (dq, dk, dv), tuple(1.05 * t + U * g.abs() + 1e-30
                               for t, g in zip((tq, tk, tv), (dq, dk, dv)))


def assert_within(got, want, tol, what=""):
    import torch
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() / tol
    assert float(over.max()) <= 1.0 if over.numel() else True, \
        f"{what}: {float(over.max()):.3f} times the tolerance"


def assert_lse(got, want, what=""):
    import torch
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: lse finiteness"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{what}: lse of empty rows"
    if fin.any():
        err = float((got[fin] - want[fin]).abs().max())
        assert err <= LSE_TOL, f"{what}: lse off by {err:.2e}"
