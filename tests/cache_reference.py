"""The 8-bit paged cache in NumPy, from its definition, for the tests."""

from __future__ import annotations

import math

import numpy as np

from exact_attention_33_gb300 import workloads as W

BLOCK = 16


def encode(x):
    """e4m3 codes of float32 values: to nearest, ties to even, infinities and
    larger values saturate, NaN stays NaN."""
    x = np.asarray(x, dtype=np.float32)
    codes = W.e4m3_encode(np.where(np.isnan(x), np.float32(0), x))
    return np.where(np.isnan(x), np.uint8(0x7F), codes)


def need_scale(amax):
    """The smallest power of two >= 2^-100 with amax <= 448 of it."""
    e = -100
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return np.float32(2.0 ** e)


def append(values, pool, scale, table, ctx, new):
    """Writes float32 `values` [T, Hkv, d] (the sequences' new tokens in a row)
    into codes `pool` [blocks, 16, Hkv, d] and `scale` [blocks, Hkv], in place."""
    a = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        first = c - n
        for blk in range(first // BLOCK, (c + BLOCK - 1) // BLOCK if n else 0):
            phys = table[b][blk]
            s0, s1 = max(0, first - blk * BLOCK), min(BLOCK, c - blk * BLOCK)
            rows = values[a + blk * BLOCK + s0 - first: a + blk * BLOCK + s1 - first]
            for h in range(pool.shape[2]):
                x = rows[:, h]
                fin = np.abs(x[np.isfinite(x)])
                s = need_scale(float(fin.max()) if fin.size else 0.0)
                if s0:
                    old = scale[phys, h]
                    s = max(s, old)
                    if s > old:
                        was = W.e4m3_decode(pool[phys, :s0, h]).astype(np.float32)
                        pool[phys, :s0, h] = encode(was * np.float32(old / s))
                pool[phys, s0:s1, h] = encode(x / s)
                scale[phys, h] = s
        a += n


def real(pool, scale):
    """What the codes stand for, float64."""
    return W.e4m3_decode(pool) * scale.astype(np.float64)[:, None, :, None]


def tables(ctx, seed, spare=3, width=None):
    """A random block table (unused entries -1) and the number of blocks."""
    blocks = [(c + BLOCK - 1) // BLOCK for c in ctx]
    perm = np.random.default_rng(seed).permutation(sum(blocks) + spare)
    table = np.full((len(ctx), max(width or 0, *blocks, 1)), -1, dtype=np.int32)
    a = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[a:a + n]
        a += n
    return table, sum(blocks) + spare


def bf16(rng, *shape):
    """Normal values, rounded to bf16, as float32."""
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32)))


# A weight is rounded to fp16 once (2^-11 of itself), the output to bf16
# (2^-8); sums, exponentials and scores are fp32 (window_reference.F).
def decode_rows(q, k, v, window, sinks, scale=None):
    """Last query row(s) q [n, d] over keys [L, d] in 64 bits: (out, lse, tol)."""
    import torch
    import window_reference as ref
    out, lse, _ = ref.forward(q, k, v, window, sinks, scale=scale)
    n, L = q.shape[0], k.shape[0]
    x = (q @ k.T) * (1.0 / math.sqrt(q.shape[1]) if scale is None else scale)
    x = x.masked_fill(~ref.visible(n, L, L - n, window, sinks, q.device), -math.inf)
    p = torch.where(lse[:, None] == -math.inf, 0.0, torch.exp(x - lse[:, None]))
    size = p @ v.abs()
    return out, lse, 1.05 * (2.0 ** -11 * size + ref.U * out.abs()) + ref.F * size + 1e-30
