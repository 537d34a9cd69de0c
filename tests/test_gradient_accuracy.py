"""How exact the windowed gradients are: a bound on their relative RMS error
that the kernels' own roundings keep and one rounding more breaks.

The kernels round dS = P (dP - D) to bf16 once, with P, dP and D = sum P dP in
fp32, and the gradient itself once.  A rounding to bf16 is off by up to 2^-8
of 2^floor(log2 x); over values whose significand m in [1, 2) has the density
1 / (m ln 2), its relative RMS is 2^-8 sqrt(E[m^-2] / 3) = 2^-8
sqrt(0.541 / 3) = 1.66e-3.  The errors of dS's terms are independent, so a sum
of many has the same relative RMS, and both roundings together sqrt(2) 1.66e-3 =
2.35e-3.  A third, of P before dS, makes 2.87e-3.  D from an output that was
rounded to bf16 makes more where few keys matter, since P (dP - D) is then a small
difference: queries four times the usual size make it 4e-3.  The bound lies between.
"""
import math

import pytest

BOUND = 2.6e-3
N, D_HEAD, WINDOW, SINKS = 700, 64, 24, 3


def rms(got, want):
    return float(((got - want).square().sum() / want.square().sum()).sqrt())


def rounded(x):
    import torch
    return x.float().to(torch.bfloat16).double()


def gradients(q, k, v, g, window, sinks, round_p=False, round_o=False, round_ds=True):
    """dq and dk [n, d] in 64 bits with bf16 roundings at the places asked for."""
    import torch
    import window_reference as ref
    n, d = q.shape
    scale = 1.0 / math.sqrt(d)
    x = (q @ k.T * scale).masked_fill(~ref.visible(n, n, 0, window, sinks, q.device), -math.inf)
    p = torch.softmax(x, 1)
    dp = g @ v.T
    D = (g * rounded(p @ v)).sum(1, keepdim=True) if round_o else (p * dp).sum(1, keepdim=True)
    ds = (rounded(p) if round_p else p) * (dp - D)
    ds = rounded(ds) if round_ds else ds
    dq, dk = scale * ds @ k, scale * ds.T @ q
    return (rounded(dq), rounded(dk)) if round_ds else (dq, dk)


def inputs(seed, *heads, device="cpu"):
    """q, k, v, g of these numbers of heads, queries of four times the usual size."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = [torch.randn(N, h, D_HEAD, generator=gen) for h in heads]
    return [t.to(torch.bfloat16).to(device) for t in (4 * x[0], *x[1:])]


def test_the_bound_tells_the_roundings_apart():
    import torch
    q, k, v, g = (t[:, 0].double() for t in inputs(1, 1, 1, 1, 1))
    exact = gradients(q, k, v, g, WINDOW, SINKS, round_ds=False)
    for more, below in ((dict(), True), (dict(round_p=True), False), (dict(round_o=True), False)):
        for got, want in zip(gradients(q, k, v, g, WINDOW, SINKS, **more), exact):
            assert (rms(got, want) <= BOUND) == below, (more, rms(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1)])
def test_gradients_round_no_more_than_stated(packed, H, Hkv):
    import torch
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa
    q, k, v, g = inputs(2, H, Hkv, Hkv, H, device="cuda")
    if packed:
        cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
        out, lse = fa.fa_fwd_varlen_window(q, k, v, cu, N, WINDOW, SINKS)
        dq, dk, _ = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, cu, N, WINDOW, SINKS)
    else:
        x = [t[None] for t in (q, k, v, g)]
        out, lse = fa.fa_fwd_window(*x[:3], WINDOW, SINKS)
        dq, dk = (t[0] for t in fa.fa_bwd_window(*x[:3], out, lse, x[3], WINDOW, SINKS)[:2])
    want_q, want_k = torch.zeros_like(q, dtype=torch.double), torch.zeros_like(k, dtype=torch.double)
    for h in range(H):
        kv = h * Hkv // H
        a, b = gradients(q[:, h].double(), k[:, kv].double(), v[:, kv].double(), g[:, h].double(),
                         WINDOW, SINKS, round_ds=False)
        want_q[:, h] = a
        want_k[:, kv] += b
    assert rms(dq.double(), want_q) <= BOUND, rms(dq.double(), want_q)
    assert rms(dk.double(), want_k) <= BOUND, rms(dk.double(), want_k)
    assert fa.fa_device_status(clear=True) == 0
