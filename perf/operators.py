"""Workloads of the windowed attention and the 8-bit cache calls.

Four operators and how a serving or training program uses them:

* windowed attention with sinks: a query at position p sees key j <= p when
  j > p - window or j < sinks.  Prompts (packed or dense), training steps
  (forward, then the gradient) and single tokens over a paged cache;
* attention over a paged cache of e4m3 codes with one scale per 16-token
  block and KV head, for single tokens and for chunks of a prompt;
* the write of new keys and values into that cache.

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it makes the library's calls.
"""

import math
import random

import torch

own = False

BLOCK = 16        # tokens of a cache block
E4M3_MAX = 448.0  # largest finite e4m3 value
MIN_EXP = -100    # smallest exponent of a block's scale


def listed():
    return [
        # a few short prompts of a small model: latency counts
        dict(name="window-prompt-short", op="window_prompt", seqs=4, lo=1, hi=97, lengths=5, H=8,
             Hkv=2, d=64, window=32, sinks=4),
        # the packed batch of ragged sequences of the benchmark, with a window
        dict(name="window-prompt-packed", op="window_prompt", seqs=32, lo=64, hi=4096, lengths=2,
             H=16, Hkv=4, d=128, window=1024, sinks=4),
        # one long prompt
        dict(name="window-prompt-long", op="window_prompt", seqs=1, lo=16384, hi=16384, lengths=1,
             H=32, Hkv=8, d=128, window=4096, sinks=64),
        # training on equal sequences, every head its own keys, no sinks, odd window
        dict(name="window-train-dense", op="window_train", seqs=4, lo=2048, hi=2048, lengths=1,
             H=16, Hkv=16, d=64, window=500, sinks=0),
        # training on packed documents with shared KV heads
        dict(name="window-train-packed", op="window_train", seqs=16, lo=1, hi=4096, lengths=3,
             H=16, Hkv=4, d=128, window=512, sinks=16),
        # one user's next token
        dict(name="window-token-one", op="window_token", batch=1, lo=5001, hi=5001, lengths=1,
             H=32, Hkv=8, d=128, window=1024, sinks=4),
        # a serving batch's next tokens, the benchmark's context lengths
        dict(name="window-token-batch", op="window_token", batch=64, lo=512, hi=32768, lengths=3,
             H=32, Hkv=8, d=128, window=4096, sinks=4),
        # the same over the 8-bit cache, every key visible
        dict(name="fp8-token-one", op="fp8_token", batch=1, lo=701, hi=701, lengths=1, H=8, Hkv=2,
             d=64, window=0, sinks=0),
        dict(name="fp8-token-batch", op="fp8_token", batch=64, lo=512, hi=32768, lengths=3, H=32,
             Hkv=8, d=128, window=0, sinks=0),
        # chunks of prompts against what the 8-bit cache holds of them
        dict(name="fp8-chunk", op="fp8_chunk", batch=4, lo=1024, hi=8192, chunk=512, lengths=6,
             H=32, Hkv=8, d=128, window=0, sinks=0),
        # the write of a serving batch's new tokens, and of whole prompts
        dict(name="fp8-append-token", op="fp8_append", batch=64, lo=17, hi=4096, new_lo=1, new_hi=1,
             lengths=4, Hkv=8, d=128),
        dict(name="fp8-append-prompt", op="fp8_append", batch=16, lo=0, hi=0, new_lo=512,
             new_hi=4096, lengths=7, Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["window_prompt", "window_prompt", "window_train", "window_token", "fp8_token",
                     "fp8_token", "fp8_chunk", "fp8_append"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 7, 8] if Hkv <= 2 else [1, 2, 4])
    case = dict(op=op, lengths=rng.randrange(1 << 20), Hkv=Hkv, d=d)
    if op != "fp8_append":
        case["H"] = H
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 0, 1, 4, 16, 64, 130])
    if op in ("window_prompt", "window_train"):
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, (32768 if op == "window_prompt" else 16384) // seqs))
        case.update(seqs=seqs, lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi, window=window,
                    sinks=sinks)
    elif op in ("window_token", "fp8_token"):
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768)
        if op == "fp8_token" and rng.random() < 0.7:
            window, sinks = 0, 0
        case.update(batch=batch, lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi, window=window,
                    sinks=sinks)
    elif op == "fp8_chunk":
        if rng.random() < 0.6:
            window, sinks = 0, 0
        hi = _log(rng, 1, 8192)
        case.update(batch=_log(rng, 1, 4), lo=rng.choice([0, hi // 4, hi]), hi=hi,
                    chunk=_log(rng, 1, 512), window=window, sinks=sinks)
    else:
        new = _log(rng, 1, 4096)
        case.update(batch=_log(rng, 1, 16), lo=0, hi=_log(rng, 1, 2048),
                    new_lo=rng.choice([1, max(1, new // 4), new]), new_hi=new)
    return case


# ------------------------------------------------------------------ lengths

def _lens(case):
    """The lengths that the case stands for (the same for every seed)."""
    r = random.Random(case["lengths"])
    n = case.get("seqs") or case["batch"]
    first = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    if case["op"] == "fp8_chunk":
        return [a + case["chunk"] for a in first], [case["chunk"]] * n
    if case["op"] == "fp8_append":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        return [a + b for a, b in zip(first, new)], new
    return first, first


def _visible(p, window, sinks):
    """Keys that a query at position p sees (window 0: every one up to p)."""
    if window <= 0:
        return p + 1
    return min(p + 1, window) + min(sinks, max(0, p + 1 - window))


def work(case):
    ctx, new = _lens(case)
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    if op == "fp8_append":
        t = sum(new)
        # keys and values read in 16 bits, their codes and the touched blocks' scales written
        touched = sum((c + BLOCK - 1) // BLOCK - (c - n) // BLOCK for c, n in zip(ctx, new))
        return {"bytes": 2 * (3 * t * Hkv * d + 4 * touched * Hkv), "flops": 4 * t * Hkv * d}
    H, window, sinks = case["H"], case["window"], case["sinks"]
    if op in ("window_prompt", "window_train"):
        t = sum(new)
        pairs = sum(_visible(p, window, sinks) for n in new for p in range(n))
        b = t * d * 2 * (2 * H + 2 * Hkv) + 4 * t * H
        if op == "window_prompt":
            return {"bytes": b, "flops": 4 * d * H * pairs}
        b += t * d * 2 * (2 * H + 2 * Hkv)  # dO read, dQ, dK and dV written
        return {"bytes": b, "flops": 14 * d * H * pairs}
    elem = 2 if op == "window_token" else 1
    if op == "fp8_chunk":
        pairs = sum(_visible(p, window, sinks) for c, n in zip(ctx, new) for p in range(c - n, c))
        # the keys that some query of the chunk sees
        keys = sum(_visible(c - 1, min(c, window + n - 1) if window else 0, sinks)
                   for c, n in zip(ctx, new))
        rows = sum(new)
    else:
        pairs = keys = sum(_visible(c - 1, window, sinks) for c in ctx)
        rows = len(ctx)
    scales = 0 if op == "window_token" else 2 * 4 * Hkv * (keys // BLOCK + len(ctx))
    b = 2 * keys * Hkv * d * elem + scales + rows * H * (4 * d + 4) + 4 * (keys // BLOCK)
    return {"bytes": b, "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------ inputs

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    ctx, new = _lens(case)
    s = dict(case=case, scale=1.0 / math.sqrt(d), window=case.get("window", 0),
             sinks=case.get("sinks", 0), max_new=max(new), max_ctx=max(ctx), kept={})
    t = sum(new)
    if op in ("window_prompt", "window_train"):
        s.update(q=normal(t, case["H"], d), k=normal(t, Hkv, d), v=normal(t, Hkv, d),
                 cu=_i32(_cu(new)), dense=case["lo"] == case["hi"])
        # a few keys stand out, as they do in trained models
        s["k"][torch.randint(0, t, (max(1, t // 100),), generator=g, device="cuda")] *= 4
        if op == "window_train":
            s["dout"] = normal(t, case["H"], d)
        return s
    # a paged cache: the blocks of all sequences in a random order, with a few free ones
    blocks = [(c + BLOCK - 1) // BLOCK for c in ctx]
    total = sum(blocks) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = _i32(_cu(blocks))[:-1, None]
    at = torch.arange(max(blocks), device="cuda", dtype=torch.int32)
    s["table"] = torch.where(at < _i32(blocks)[:, None], perm[(first + at).clamp(max=total - 1)], -1)
    s["table"] = s["table"].to(torch.int32).contiguous()
    s["ctx"], s["cu"] = _i32(ctx), _i32(_cu(new))
    if op == "window_token":
        s.update(q=normal(len(ctx), case["H"], d), k_pool=normal(total, BLOCK, Hkv, d),
                 v_pool=normal(total, BLOCK, Hkv, d))
        return s
    for x in ("k", "v"):
        # each block's largest magnitude differs, and so does its scale
        exp = torch.randint(-9, -5, (total, Hkv), generator=g, device="cuda")
        unit = normal(total, BLOCK, Hkv, d).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX)
        s[x + "_pool"] = unit.to(torch.float8_e4m3fn)
        s[x + "_scale"] = torch.ldexp(torch.ones((), device="cuda"), exp)
        del unit
    if op == "fp8_append":
        s.update(k=normal(t, Hkv, d), v=normal(t, Hkv, d))
        s["v"] *= 3
    else:
        s["q"] = normal(len(ctx) if op == "fp8_token" else t, case["H"], d)
    return s


# ------------------------------------------------------------------ plain forms

def _softmax_parts(scores, mask):
    """exp(s - max), its row sums and the log-sum-exp over the last axis."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e, total, (top + torch.log(total)).squeeze(-1)


def _plain_prompt(s, q, k, v):
    """Windowed attention of packed 32-bit tensors, by blocks of queries: each
    block's keys are gathered from its first window's start to its last row;
    the sinks of all sequences are further columns."""
    T, H, d = q.shape
    Hkv = k.shape[1]
    W, sinks = min(s["window"], s["max_new"]), min(s["sinks"], s["max_new"])
    cu = s["cu"].long()
    C = min(256, T)
    nb = (T + C - 1) // C
    dev = q.device
    row = torch.arange(nb * C, device=dev)
    rowc = row.clamp(max=T - 1)
    seq = torch.searchsorted(cu, rowc, right=True) - 1
    start = cu[seq]
    qb = q.index_select(0, rowc).view(nb, C, Hkv, H // Hkv, d)
    key = torch.arange(nb, device=dev)[:, None] * C + torch.arange(-(W - 1), C, device=dev)
    at = key.clamp(0, T - 1).flatten()
    kb = k.index_select(0, at).view(nb, -1, Hkv, d)  # [nb, L, Hkv, d]
    vb = v.index_select(0, at).view(nb, -1, Hkv, d)
    r = row.view(nb, C, 1)
    mask = (key[:, None] <= r) & (key[:, None] > r - W) & (key[:, None] >= start.view(nb, C, 1))
    scores = torch.einsum("nchgd,nlhd->nhgcl", qb, kb)
    mask = mask[:, None, None]
    if sinks:
        sk = (cu[:-1, None] + torch.arange(sinks, device=dev)).flatten()
        owner = torch.arange(cu.numel() - 1, device=dev).repeat_interleave(sinks)
        ks, vs = (x.index_select(0, sk.clamp(max=T - 1)) for x in (k, v))
        sm = (owner == seq.view(nb, C, 1)) & (sk <= r - W)
        scores = torch.cat([scores, torch.einsum("nchgd,lhd->nhgcl", qb, ks)], -1)
        mask = torch.cat([mask, sm[:, None, None]], -1)
    e, total, lse = _softmax_parts(scores * s["scale"], mask)
    L = kb.shape[1]
    out = torch.einsum("nhgcl,nlhd->nchgd", e[..., :L], vb)
    if sinks:
        out = out + torch.einsum("nhgcl,lhd->nchgd", e[..., L:], vs)
    out = out / total.permute(0, 3, 1, 2, 4)
    out, lse = out.reshape(nb * C, H, d)[:T], lse.permute(1, 2, 0, 3).reshape(H, nb * C)[:, :T]
    if s["dense"]:
        B = s["case"]["seqs"]
        return out.view(B, -1, H, d), lse.view(H, B, -1).transpose(0, 1)
    return out, lse


def _batch(s, x):
    """A packed tensor as the dense call's where all sequences have one length."""
    return x.view(s["case"]["seqs"], -1, *x.shape[1:]) if s["dense"] else x


def _plain_pages(s, pool, scale, slots):
    """Values of the cache's tokens `slots`, in 32 bits."""
    x = pool.view(-1, *pool.shape[2:])
    if scale is None:
        return x[slots].float()
    codes = x.view(torch.uint8)[slots].view(torch.float8_e4m3fn).float()
    return codes * scale[slots // BLOCK][..., None]


def _plain_cached(s, k_scale=None, v_scale=None):
    """Queries (the last rows of each sequence) against a paged cache: the
    sequences are padded to the longest."""
    q, ctx, cu = s["q"], s["ctx"].long(), s["cu"].long()
    H, d = q.shape[1:]
    Hkv = s["k_pool"].shape[2]
    S, dev = ctx.numel(), q.device
    nq = s["max_new"] if s["case"]["op"] == "fp8_chunk" else 1
    n = (cu[1:] - cu[:-1]) if nq > 1 else torch.ones_like(ctx)
    W, sinks, longest = s["window"], s["sinks"], s["max_ctx"]
    if W and W + nq + sinks < longest:  # only the sinks and the windows of the rows
        low = (ctx - n - W + 1).clamp(min=0)
        pos = low[:, None] + torch.arange(W + nq - 1, device=dev)
        sink = torch.arange(sinks, device=dev).expand(S, sinks)
        pos = torch.cat([torch.where(sink < low[:, None], sink, longest), pos], 1)
    else:
        pos = torch.arange(longest, device=dev).expand(S, longest)
    inside = pos < ctx[:, None]
    blk = torch.gather(s["table"].long(), 1, (pos // BLOCK).clamp(max=s["table"].shape[1] - 1))
    slots = (blk.clamp(min=0) * BLOCK + pos % BLOCK)
    k = _plain_pages(s, s["k_pool"], k_scale, slots)
    row = torch.arange(nq, device=dev)
    qi = ((cu[:-1] if nq > 1 else torch.arange(S, device=dev))[:, None] + row).clamp(max=q.shape[0] - 1)
    qp = q.float()[qi].view(S, nq, Hkv, H // Hkv, d)
    at = (ctx - n)[:, None] + row  # each query's position
    mask = inside[:, None] & (pos[:, None] <= at[..., None])
    if W:
        mask &= (pos[:, None] > at[..., None] - W) | (pos[:, None] < sinks)
    scores = torch.einsum("sqhgd,slhd->shgql", qp, k) * s["scale"]
    del k
    e, total, lse = _softmax_parts(scores, mask[:, None, None])
    v = _plain_pages(s, s["v_pool"], v_scale, slots)
    out = torch.einsum("shgql,slhd->sqhgd", e, v) / total.permute(0, 3, 1, 2, 4)
    if nq == 1:
        return {"out": out.reshape(S, H, d).to(torch.bfloat16), "lse": lse.reshape(S, H)}
    # every chunk of a case has the same length
    return {"out": out.reshape(S * nq, H, d).to(torch.bfloat16),
            "lse": lse.permute(1, 2, 0, 3).reshape(H, S * nq)}


def _plain_append(s):
    ctx, cu, table = s["ctx"].long(), s["cu"].long(), s["table"].long()
    T = s["k"].shape[0]
    dev = table.device
    first = ctx - (cu[1:] - cu[:-1])  # position of each sequence's first new token
    tok = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = first[seq] + tok - cu[seq]
    block, slot = table[seq, pos // BLOCK], pos % BLOCK
    head = table.gather(1, (first // BLOCK)[:, None])[:, 0]  # each sequence's first written block
    begun = first % BLOCK                                    # tokens it held before
    for x in ("k", "v"):
        pool, scale, new = s[x + "_pool"], s[x + "_scale"], s[x].float()
        codes = pool.view(torch.uint8)
        amax = torch.zeros_like(scale)
        amax.index_reduce_(0, block, new.abs().amax(-1), "amax")
        m, e = torch.frexp(amax)  # amax = m 2^e, m of [0.5, 1); 448 = 0.875 2^9
        e = torch.where(m <= 0.875, e - 9, e - 8)
        e = torch.where(amax == 0, MIN_EXP, e).clamp(min=MIN_EXP)
        need = torch.ldexp(torch.ones_like(amax), e)
        before = torch.where(begun[:, None] > 0, scale[head], 0.0)
        after = torch.maximum(before, need[head])
        kept = pool.view(torch.uint8)[head].view(torch.float8_e4m3fn).float()
        again = (kept * (before / after)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        old = torch.arange(BLOCK, device=dev) < begun[:, None]
        codes[head] = torch.where(old[..., None, None], again, codes[head])
        scale[block] = need[block]
        scale[head] = after
        codes[block, slot] = (new / scale[block][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return _cache(s)


def _cache(s):
    return {x: s[x] for x in ("k_pool", "v_pool", "k_scale", "v_scale")}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "window_prompt":
        out, lse = _plain_prompt(s, s["q"].float(), s["k"].float(), s["v"].float())
        return {"out": out.to(torch.bfloat16), "lse": lse}
    if op == "window_train":
        x = [s[n].float().requires_grad_() for n in ("q", "k", "v")]
        out, lse = _plain_prompt(s, *x)
        grads = torch.autograd.grad(out, x, _batch(s, s["dout"]).float())
        return {"out": out.detach().to(torch.bfloat16), "lse": lse.detach(),
                **{n: _batch(s, t.to(torch.bfloat16)) for n, t in zip(("dq", "dk", "dv"), grads)}}
    if op == "fp8_append":
        return _plain_append(s)
    if op == "window_token":
        return _plain_cached(s)
    return _plain_cached(s, s["k_scale"], s["v_scale"])


def _run_own(s, op):
    import exact_attention_33_gb300 as fa
    case, kept = s["case"], s["kept"]
    H, Hkv, d = case.get("H"), case["Hkv"], case["d"]
    W, sinks = s["window"], s["sinks"]
    if op in ("window_prompt", "window_train"):
        q, k, v = (_batch(s, s[n]) for n in ("q", "k", "v"))
        if s["dense"]:  # sequences of one length: the dense call
            out, lse = fa.fa_fwd_window(q, k, v, W, sinks)
        else:
            out, lse = fa.fa_fwd_varlen_window(q, k, v, s["cu"], s["max_new"], W, sinks)
        grads = {}
        if op == "window_train":
            if "workspace" not in kept:
                size = fa.fa_bwd_window_workspace_size(case["seqs"], H, Hkv, s["max_new"], d, W,
                                                       sinks)
                kept["workspace"] = fa.new_workspace(size)
            if s["dense"]:
                g = fa.fa_bwd_window(q, k, v, out, lse, _batch(s, s["dout"]), W, sinks,
                                     workspace=kept["workspace"])
            else:
                g = fa.fa_bwd_varlen_window(q, k, v, out, lse, s["dout"], s["cu"], s["max_new"], W,
                                            sinks, workspace=kept["workspace"])
            grads = dict(zip(("dq", "dk", "dv"), g))
        return {"out": out, "lse": lse, **grads}
    if op == "fp8_append":
        fa.fa_cache_append_fp8(s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"],
                               s["v_scale"], s["table"], s["ctx"], s["cu"], s["max_new"])
        return _cache(s)
    if op == "fp8_chunk":
        out, lse = fa.fa_fwd_paged_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                       s["table"], s["ctx"], s["cu"], s["max_new"], s["max_ctx"],
                                       window=W, sinks=sinks)
        return {"out": out, "lse": lse}
    if "workspace" not in kept:
        kept["workspace"] = fa.new_workspace(fa.fa_decode_window_workspace_size(
            case["batch"], H, Hkv, d, s["max_ctx"], W, sinks))
    if op == "window_token":
        out, lse = fa.fa_decode_paged_window(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx"],
                                             s["max_ctx"], W, sinks, workspace=kept["workspace"])
    else:
        out, lse = fa.fa_decode_paged_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"],
                                          s["v_scale"], s["table"], s["ctx"], s["max_ctx"],
                                          window=W, sinks=sinks, workspace=kept["workspace"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ 64 bits

def _rows_exact(q, k, v, first, window, sinks, dout=None):
    """Rows q [n, d] at positions first, first + 1, ... over keys [L, d], all
    float64, from the definition: (out, lse) and, with dout, (dq, dk, dv)."""
    n, d = q.shape
    L = k.shape[0]
    i = first + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)
    hidden = j > i
    if window:
        hidden |= (j <= i - window) & (j >= sinks)
    x = q @ k.T / math.sqrt(d)
    x[hidden] = -math.inf
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    out = p @ v
    if dout is None:
        return out, lse
    dp = dout @ v.T
    ds = p * (dp - (dout * out).sum(1, keepdim=True)) / math.sqrt(d)
    return out, lse, ds @ k, ds.T @ q, p.T @ dout


def exact(case, seed):
    s = prepare(case, seed)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    ctx, new = _lens(case)
    if op == "fp8_append":
        return _exact_append(s, ctx, new)
    H, W, sinks = case["H"], s["window"], s["sinks"]
    G = H // Hkv
    rows = [1] * len(ctx) if op in ("window_token", "fp8_token") else new
    # about 1e12 products in 64 bits a second and less
    if sum(n * c for n, c in zip(rows, ctx)) * H * d * (4 if op != "window_train" else 10) > 6e12:
        return None
    q = s["q"].double()
    lse = torch.empty(H, q.shape[0], dtype=torch.float64, device="cuda")
    out = torch.empty_like(q)
    if op in ("window_prompt", "window_train"):
        k, v = s["k"].double(), s["v"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        a = 0
        for n in new:
            at = slice(a, a + n)
            for h in range(H):
                got = _rows_exact(q[at, h], k[at, h // G], v[at, h // G], 0, W, sinks,
                                  s["dout"][at, h].double() if op == "window_train" else None)
                out[at, h], lse[h, at] = got[:2]
                if op == "window_train":
                    dq[at, h] = got[2]
                    dk[at, h // G] += got[3]
                    dv[at, h // G] += got[4]
            a += n
        if s["dense"]:
            lse = lse.view(H, len(new), -1).transpose(0, 1)
        grads = dict(dq=dq, dk=dk, dv=dv) if op == "window_train" else {}
        return {"lse": lse, **{n: _batch(s, x) for n, x in dict(out=out, **grads).items()}}
    a = 0
    for b, c in enumerate(ctx):
        n = rows[b]
        pages = s["table"][b, : (c + BLOCK - 1) // BLOCK].long()
        kv = []
        for x in ("k", "v"):
            t = s[x + "_pool"][pages].double() if op == "window_token" else (
                s[x + "_pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
                * s[x + "_scale"][pages].double()[:, None, :, None])
            kv.append(t.flatten(0, 1)[:c])
        for h in range(Hkv):
            # the group's heads share the keys: one call on their rows, head by head
            for g in range(G):
                at = slice(a, a + n)
                got = _rows_exact(q[at, h * G + g], kv[0][:, h], kv[1][:, h], c - n, W, sinks)
                out[at, h * G + g], lse[h * G + g, at] = got
        a += n
    return {"out": out, "lse": lse if op == "fp8_chunk" else lse.T.contiguous()}


def _e4m3(x):
    """Nearest e4m3 value of each float64 value (ties to the even code)."""
    size = x.abs().clamp(max=E4M3_MAX)
    exp = torch.floor(torch.log2(size.clamp(min=2.0 ** -6)))
    step = torch.exp2(exp - 3)
    return torch.copysign(torch.round(size / step) * step, x)


def _exact_append(s, ctx, new):
    got = {}
    for x in ("k", "v"):
        codes = s[x + "_pool"].double()
        scale = s[x + "_scale"].double()
        values = s[x].double()
        a = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            f = c - n
            lo, hi = f // BLOCK, (c + BLOCK - 1) // BLOCK
            pages = s["table"][b, lo:hi].long()
            # the tokens of these blocks in a row, from the first block's first slot
            rows = torch.zeros((hi - lo) * BLOCK, *values.shape[1:], dtype=torch.float64, device="cuda")
            rows[f - lo * BLOCK: c - lo * BLOCK] = values[a:a + n]
            rows = rows.view(hi - lo, BLOCK, *values.shape[1:])
            amax = rows.abs().amax((1, 3))
            # the smallest power of two with amax <= 448 need; log2 may be one off at borders
            need = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(min=MIN_EXP))
            need = torch.where(need * E4M3_MAX < amax, need * 2, need)
            need = torch.where((need / 2 * E4M3_MAX >= amax) & (need > 2.0 ** MIN_EXP), need / 2, need)
            old = f - lo * BLOCK
            if old:
                before = scale[pages[0]].clone()
                need[0] = torch.maximum(need[0], before)
                codes[pages[0], :old] = _e4m3(codes[pages[0], :old] * (before / need[0])[None, :, None])
            fresh = _e4m3(rows / need[:, None, :, None])
            where = torch.arange((hi - lo) * BLOCK, device="cuda").view(hi - lo, BLOCK)
            mine = (where >= old) & (where < c - lo * BLOCK)
            codes[pages] = torch.where(mine[..., None, None], fresh, codes[pages])
            scale[pages] = need
            a += n
        got[x + "_pool"], got[x + "_scale"] = codes, scale
    return got
