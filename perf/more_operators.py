"""Workloads of the rotary positions, of the cache writes that apply them, and
of decoding over shared prefixes.

Three operators, in the order in which a program meets them:

* rotation of queries and keys by their positions, over whole heads or the
  first part of each, in the half and the interleaved layout, at scaled
  frequencies; for training the rotation of the gradients too;
* the write of new keys and values into a paged cache (bf16, or e4m3 codes
  with a scale per block and head) with the rotation on the way, which rotates
  the queries as well;
* single tokens of a batch in which groups of sequences share a long prefix,
  whose cache blocks serve the whole group.

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits (angles in 64); with ``own`` true it makes the library's calls.
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
        dict(name="rope-prompt-short", op="rope", seqs=4, lo=1, hi=97, lengths=5, start=0, H=8, Hkv=2,
             d=64, rot=64, interleaved=False, base=10000.0, stretch=1.0, train=False),
        # a training step on the benchmark's packed batch: q and k, then their gradients
        dict(name="rope-train-packed", op="rope", seqs=32, lo=64, hi=4096, lengths=2, start=0, H=16,
             Hkv=4, d=128, rot=128, interleaved=False, base=10000.0, stretch=1.0, train=True),
        # the benchmark's long dense prompts; half of each head, stretched for long contexts
        dict(name="rope-dense-long", op="rope", seqs=2, lo=8192, hi=8192, lengths=1, start=0, H=32,
             Hkv=32, d=128, rot=64, interleaved=True, base=500000.0, stretch=8.0, train=False),
        # a serving batch's next tokens into the bf16 cache
        dict(name="append-token", op="append", batch=64, lo=17, hi=4096, new_lo=1, new_hi=1,
             lengths=4, H=32, Hkv=8, d=128, rot=128, interleaved=False, base=500000.0, stretch=1.0),
        # chunks of prompts behind what the cache holds, an odd group of heads, a rotated quarter
        dict(name="append-chunk", op="append", batch=5, lo=0, hi=2000, new_lo=1, new_hi=300,
             lengths=6, H=14, Hkv=2, d=64, rot=16, interleaved=True, base=10000.0, stretch=1.0),
        # whole prompts
        dict(name="append-prompt", op="append", batch=16, lo=0, hi=0, new_lo=512, new_hi=4096,
             lengths=7, H=32, Hkv=8, d=128, rot=128, interleaved=False, base=500000.0, stretch=8.0),
        # the same two, tokens and prompts, into the 8-bit cache
        dict(name="append8-token", op="append8", batch=64, lo=17, hi=4096, new_lo=1, new_hi=1,
             lengths=4, H=32, Hkv=8, d=128, rot=128, interleaved=False, base=500000.0, stretch=1.0),
        dict(name="append8-prompt", op="append8", batch=16, lo=0, hi=0, new_lo=512, new_hi=4096,
             lengths=7, H=32, Hkv=8, d=128, rot=128, interleaved=False, base=500000.0, stretch=1.0),
        # a few users of a small model with one system prompt
        dict(name="prefix-few", op="prefix", batch=3, idle=0, groups=1, lo=1001, hi=1001, own_lo=1,
             own_hi=40, lengths=8, H=8, Hkv=2, d=64),
        # a serving batch over one long document
        dict(name="prefix-batch", op="prefix", batch=64, idle=0, groups=1, lo=8192, hi=8192, own_lo=1,
             own_hi=1024, lengths=9, H=32, Hkv=8, d=128),
        # four prompts of different lengths in a batch padded with idle slots
        dict(name="prefix-groups", op="prefix", batch=64, idle=3, groups=4, lo=512, hi=32768,
             own_lo=16, own_hi=2048, lengths=11, H=32, Hkv=8, d=128),
        # many samples of one long prompt: the products count
        dict(name="prefix-many", op="prefix", batch=256, idle=0, groups=1, lo=16384, hi=16384,
             own_lo=1, own_hi=512, lengths=12, H=32, Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append8", "prefix", "prefix"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 7, 8] if Hkv <= 2 else [1, 2, 4])
    case = dict(op=op, lengths=rng.randrange(1 << 20), H=H, Hkv=Hkv, d=d)
    if op == "prefix":
        groups = rng.choice([1, 1, 1, 2, 3, 7])
        batch = max(groups, _log(rng, 1, 128))
        hi = _log(rng, 1, 16384)
        own_hi = _log(rng, 1, 1024)
        case.update(batch=batch, idle=rng.choice([0, 0, min(2, batch - 1)]), groups=groups,
                    lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi,
                    own_lo=rng.choice([1, max(1, own_hi // 4), own_hi]), own_hi=own_hi)
        return case
    case.update(rot=rng.choice([d, d, d // 2, d // 4, d - 16]), interleaved=rng.random() < 0.4,
                base=rng.choice([10000.0, 500000.0]), stretch=rng.choice([1.0, 1.0, 2.0, 8.0, 32.0]))
    if op == "rope":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, 32768 // seqs))
        case.update(seqs=seqs, lo=rng.choice([1, max(1, hi // 4), hi]), hi=hi,
                    start=rng.choice([0, _log(rng, 1, 1 << 20)]), train=rng.random() < 0.5)
        if case["lo"] == hi:
            case["start"] = 0
    else:
        new = _log(rng, 1, 4096)
        case.update(batch=_log(rng, 1, 16 if new > 64 else 64), lo=0, hi=_log(rng, 1, 2048),
                    new_lo=rng.choice([1, max(1, new // 4), new]), new_hi=new)
    return case


# ------------------------------------------------------------------ lengths

def _lens(case):
    """The lengths that the case stands for (the same for every seed): rope
    (lengths), cache writes (context lengths, new tokens), prefixes (context
    lengths, each group's prefix, the groups' first sequences)."""
    r = random.Random(case["lengths"])
    if case["op"] == "rope":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n = case["batch"]
    if case["op"] != "prefix":
        first = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        return [a + b for a, b in zip(first, new)], new
    shared = [r.randint(case["lo"], case["hi"]) for _ in range(case["groups"])]
    cuts = sorted(r.sample(range(1, n), case["groups"] - 1))
    cu = [0, *cuts, n]
    ctx = [shared[g] + r.randint(case["own_lo"], case["own_hi"])
           for g in range(case["groups"]) for _ in range(cu[g], cu[g + 1])]
    for b in range(n - case["idle"], n):  # padded slots hold no sequence
        ctx[b] = 0
    return ctx, shared, cu


def work(case):
    op, H, Hkv, d = case["op"], case["H"], case["Hkv"], case["d"]
    if op == "rope":
        t = sum(_lens(case)) * (2 if case["train"] else 1)
        return {"bytes": 4 * t * (H + Hkv) * d, "flops": 3 * t * (H + Hkv) * case["rot"]}
    if op == "prefix":
        ctx, shared, cu = _lens(case)
        keys = 0  # read once for a group, and each sequence's own
        for g, p in enumerate(shared):
            p = p // BLOCK * BLOCK
            keys += p + sum(max(0, c - p) for c in ctx[cu[g]:cu[g + 1]])
        return {"bytes": 4 * keys * Hkv * d + len(ctx) * H * (4 * d + 4) + 4 * (keys // BLOCK),
                "flops": 4 * d * H * sum(ctx)}
    ctx, new = _lens(case)
    t = sum(new)
    if op == "append":
        return {"bytes": 4 * t * (H + 2 * Hkv) * d, "flops": 3 * t * (H + Hkv) * case["rot"]}
    # keys and values read in 16 bits, their codes and the touched blocks' scales written
    touched = sum((c + BLOCK - 1) // BLOCK - (c - n) // BLOCK for c, n in zip(ctx, new))
    return {"bytes": 4 * t * H * d + 2 * (3 * t * Hkv * d + 4 * touched * Hkv),
            "flops": 3 * t * (H + Hkv) * case["rot"] + 4 * t * Hkv * d}


# ------------------------------------------------------------------ inputs

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _frequencies(rot, base, stretch):
    """Radians a position for each pair, and the factor of the rotated values:
    with a stretch, pairs that turn less than once over 8192 positions are
    slowed by it, those that turn over 32 times are not."""
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if stretch == 1.0:
        return freq, 1.0
    keep = [min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 31.0)) for f in freq]
    return [f * w + f / stretch * (1 - w) for f, w in zip(freq, keep)], 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    op, H, Hkv, d = case["op"], case["H"], case["Hkv"], case["d"]
    s = dict(case=case, kept={})
    if op != "prefix":
        freq, s["factor"] = _frequencies(case["rot"], case["base"], case["stretch"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["interleaved"] = case["interleaved"]
    if op == "rope":
        lens = _lens(case)
        dense = case["lo"] == case["hi"]
        shape = (len(lens), lens[0]) if dense else (sum(lens),)
        s.update(q=normal(*shape, H, d), k=normal(*shape, Hkv, d), positions=None)
        if not dense:
            s["positions"] = _i32([case["start"] + i for n in lens for i in range(n)])
        if case["train"]:
            s.update(dq=normal(*shape, H, d), dk=normal(*shape, Hkv, d))
        return s
    ctx, rest = _lens(case)[:2]
    shared, cu = [0], [0, len(ctx)]
    if op == "prefix":
        _, shared, cu = _lens(case)
    # a paged cache: the blocks of all sequences in a random order, with a few free ones; the
    # sequences of a group begin with the same whole blocks
    rows, total = [], 0
    for a, e, p in zip(cu, cu[1:], shared):
        common = list(range(total, total + p // BLOCK))
        total += len(common)
        for b in range(a, e):
            mine = max(0, (ctx[b] + BLOCK - 1) // BLOCK - len(common))
            rows.append(common + list(range(total, total + mine)))
            total += mine
    perm = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(len(r) for r in rows))
    at = torch.tensor([r + [-1] * (width - len(r)) for r in rows], device="cuda")
    s["table"] = torch.where(at >= 0, perm[at.clamp(min=0)], -1).to(torch.int32).contiguous()
    s["ctx"] = _i32(ctx)
    total += 3
    if op == "append8":
        for x in ("k", "v"):
            # each block's largest magnitude differs, and so does its scale
            exp = torch.randint(-9, -5, (total, Hkv), generator=g, device="cuda")
            unit = normal(total, BLOCK, Hkv, d).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX)
            s[x + "_pool"] = unit.to(torch.float8_e4m3fn)
            s[x + "_scale"] = torch.ldexp(torch.ones_like(exp, dtype=torch.float32), exp)
            del unit
    else:
        s.update(k_pool=normal(total, BLOCK, Hkv, d), v_pool=normal(total, BLOCK, Hkv, d))
    if op == "prefix":
        # a few keys stand out, as they do in trained models
        s["k_pool"].view(-1, Hkv, d)[
            torch.randint(0, total * BLOCK, (max(1, total // 6),), generator=g, device="cuda")] *= 4
        s.update(q=normal(len(ctx), H, d), shared=_i32(shared), groups=_i32(cu),
                 scale=1.0 / math.sqrt(d), max_shared=max(shared),
                 max_own=max(max(0, c - p) for a, e, p in zip(cu, cu[1:], shared)
                             for c in ctx[a:e]),
                 max_group=max(e - a for a, e in zip(cu, cu[1:])))
        return s
    t = sum(rest)
    # q, k and v come out of one projection, the heads of a token side by side
    qkv = normal(t, H + 2 * Hkv, d)
    s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], new=_i32(_cu(rest)),
             max_new=max(rest))
    return s


# ------------------------------------------------------------------ plain forms

def _turn(x, positions, s, back=False):
    """Rows x [..., heads, d] in 32 bits, rotated by their positions [...]."""
    angle = positions.double()[..., None] * s["freq"]
    cos = (torch.cos(angle) * s["factor"]).float()[..., None, :]
    sin = (torch.sin(angle) * s["factor"]).float()[..., None, :]
    if back:
        sin = -sin
    r = s["freq"].numel()
    if s["interleaved"]:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., 2 * r:]], -1)


def _plain_rope(s):
    q, k, at = s["q"], s["k"], s["positions"]
    if at is None:
        at = torch.arange(q.shape[-3], device=q.device).expand(q.shape[:-2])
    got = {n: _turn(x.float(), at, s).to(torch.bfloat16) for n, x in (("q", q), ("k", k))}
    if s["case"]["train"]:
        got.update({n: _turn(s[n].float(), at, s, back=True).to(torch.bfloat16)
                    for n in ("dq", "dk")})
    return got


def _slots(s):
    """Position, cache block and slot of each new token."""
    ctx, cu, table = s["ctx"].long(), s["new"].long(), s["table"].long()
    tok = torch.arange(s["k"].shape[0], device=table.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = (ctx - (cu[1:] - cu[:-1]))[seq] + tok - cu[seq]
    return pos, table[seq, pos // BLOCK], pos % BLOCK


def _plain_append(s):
    pos, block, slot = _slots(s)
    s["k_pool"][block, slot] = _turn(s["k"].float(), pos, s).to(torch.bfloat16)
    s["v_pool"][block, slot] = s["v"]
    return {"q": _turn(s["q"].float(), pos, s).to(torch.bfloat16), **_cache(s)}


def _plain_append8(s):
    pos, block, slot = _slots(s)
    ctx, cu, table = s["ctx"].long(), s["new"].long(), s["table"].long()
    first = ctx - (cu[1:] - cu[:-1])
    head = table.gather(1, (first // BLOCK)[:, None])[:, 0]  # each sequence's first written block
    begun = first % BLOCK                                    # tokens it held before
    for x, grow in (("k", max(1.0, math.sqrt(2.0) * s["factor"])), ("v", 1.0)):
        pool, scale, new = s[x + "_pool"], s[x + "_scale"], s[x].float()
        codes = pool.view(torch.uint8)
        amax = torch.zeros_like(scale)
        amax.index_reduce_(0, block, new.abs().amax(-1), "amax")
        # a rotation grows no value by more than this
        m, e = torch.frexp(amax * torch.tensor(grow, dtype=torch.float32, device=amax.device))
        e = torch.where(m <= 0.875, e - 9, e - 8)  # m 2^e with m of [0.5, 1); 448 = 0.875 2^9
        e = torch.where(amax == 0, MIN_EXP, e).clamp(min=MIN_EXP)
        need = torch.ldexp(torch.ones_like(amax), e)
        before = torch.where(begun[:, None] > 0, scale[head], 0.0)
        after = torch.maximum(before, need[head])
        kept = pool.view(torch.uint8)[head].view(torch.float8_e4m3fn).float()
        again = (kept * (before / after)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        old = torch.arange(BLOCK, device=begun.device) < begun[:, None]
        codes[head] = torch.where(old[..., None, None], again, codes[head])
        scale[block] = need[block]
        scale[head] = after
        if x == "k":
            new = _turn(new, pos, s)
        code = (new / scale[block][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        codes[block, slot] = code.view(torch.uint8)
    return {"q": _turn(s["q"].float(), pos, s).to(torch.bfloat16), **_cache(s)}


def _cache(s):
    return {x: s[x] for x in ("k_pool", "v_pool", "k_scale", "v_scale") if x in s}


def _plain_prefix(s):
    """Scores of the groups' shared blocks by one product for each group, those
    of each sequence's own keys beside them."""
    q, ctx, cu = s["q"].float(), s["ctx"].long(), s["groups"].long()
    B, H, d = q.shape
    Hkv = s["k_pool"].shape[2]
    dev = q.device
    whole = s["shared"].long() // BLOCK * BLOCK
    b = torch.arange(B, device=dev)
    g = torch.searchsorted(cu, b, right=True) - 1
    lead, table = cu[:-1], s["table"].long()
    # members of each group, padded to the largest
    rows = (lead[:, None] + torch.arange(s["max_group"], device=dev)).clamp(max=B - 1)

    def pages(pool, table, pos):
        blk = table.gather(1, (pos // BLOCK).clamp(max=table.shape[1] - 1)).clamp(min=0)
        return pool.view(-1, Hkv, d)[blk * BLOCK + pos % BLOCK].float()

    P = s["max_shared"] // BLOCK * BLOCK
    first = torch.arange(P, device=dev).expand(len(lead), P)
    mine = whole[g][:, None] + torch.arange(s["max_own"] + BLOCK - 1, device=dev)
    qh = q.view(B, Hkv, H // Hkv, d)
    x = torch.einsum("nmhgd,nphd->nmhgp", qh[rows], pages(s["k_pool"], table[lead], first))
    x = torch.cat([x[g, b - lead[g]],
                   torch.einsum("bhgd,blhd->bhgl", qh, pages(s["k_pool"], table, mine))], -1)
    seen = torch.cat([first[g] < torch.minimum(whole[g], ctx)[:, None], mine < ctx[:, None]], 1)
    x = (x * s["scale"]).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("nmhgp,nphd->nmhgd", e[..., :P][rows], pages(s["v_pool"], table[lead], first))
    out = out[g, b - lead[g]] + torch.einsum("bhgl,blhd->bhgd", e[..., P:],
                                             pages(s["v_pool"], table, mine))
    out = torch.where(total > 0, out / total, 0.0)
    return {"out": out.reshape(B, H, d).to(torch.bfloat16),
            "lse": (top + torch.log(total)).reshape(B, H)}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "rope":
        return _plain_rope(s)
    if op == "append":
        return _plain_append(s)
    if op == "append8":
        return _plain_append8(s)
    return _plain_prefix(s)


def _run_own(s, op):
    import exact_attention_33_gb300 as fa
    if op == "prefix":
        kept, (B, H, d) = s["kept"], s["q"].shape
        if "workspace" not in kept:
            kept["workspace"] = fa.new_workspace(fa.fa_decode_prefix_workspace_size(
                B, H, s["case"]["Hkv"], d, s["max_shared"], s["max_own"]))
        out, lse = fa.fa_decode_paged_prefix(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx"],
                                             s["groups"], s["shared"], s["max_shared"], s["max_own"],
                                             workspace=kept["workspace"])
        return {"out": out, "lse": lse}
    turn = dict(factor=s["factor"], interleaved=s["interleaved"])
    if op == "rope":
        q, k = fa.fa_rope(s["q"], s["k"], s["freq"], s["positions"], **turn)
        if not s["case"]["train"]:
            return {"q": q, "k": k}
        dq, dk = fa.fa_rope_bwd(s["dq"], s["dk"], s["freq"], s["positions"], **turn)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    if op == "append":
        q = fa.fa_cache_append_rope(s["q"], s["k"], s["v"], s["freq"], s["k_pool"], s["v_pool"],
                                    s["table"], s["ctx"], s["new"], s["max_new"], **turn)
    else:
        q = fa.fa_cache_append_rope_fp8(s["q"], s["k"], s["v"], s["freq"], s["k_pool"], s["v_pool"],
                                        s["k_scale"], s["v_scale"], s["table"], s["ctx"], s["new"],
                                        s["max_new"], **turn)
    return {"q": q, **_cache(s)}


# ------------------------------------------------------------------ 64 bits

def _rotated(x, first, s, back=False):
    """Rows x [n, heads, d] at positions first, first + 1, ..., by complex products in 64 bits."""
    x = x.double()
    n, r = x.shape[0], s["freq"].numel()
    p = torch.arange(first, first + n, dtype=torch.float64, device=x.device)
    w = torch.polar(torch.full((n, r), float(s["factor"]), dtype=torch.float64, device=x.device),
                    torch.outer(p, s["freq"]))
    if back:
        w = w.conj()
    head = x[..., :2 * r].unflatten(-1, (r, 2) if s["interleaved"] else (2, r))
    if not s["interleaved"]:
        head = head.transpose(-1, -2)
    z = torch.view_as_complex(head.contiguous()) * w[:, None]
    y = torch.view_as_real(z)
    if not s["interleaved"]:
        y = y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., 2 * r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefix":
        return _exact_prefix(s, case)
    if op == "rope":
        lens = _lens(case)
        got = {}
        for name in ("q", "k") + (("dq", "dk") if case["train"] else ()):
            x = s[name].flatten(0, 1) if s["positions"] is None else s[name]
            y = torch.cat([_rotated(part, case["start"], s, back=name[0] == "d")
                           for part in x.split(lens)])
            got[name] = y.view(s[name].shape)
        return got
    ctx, new = _lens(case)
    q = torch.cat([_rotated(x, c - n, s) for x, c, n in zip(s["q"].split(new), ctx, new)])
    pools = {x: s[x].double() for x in ("k_pool", "v_pool", "k_scale", "v_scale") if x in s}
    a = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        f = c - n
        lo, hi = f // BLOCK, (c + BLOCK - 1) // BLOCK
        pages = s["table"][b, lo:hi].long()
        old = f - lo * BLOCK
        for x in ("k", "v"):
            fresh, raw = s[x][a:a + n], s[x][a:a + n].double()
            fresh = _rotated(fresh, f, s) if x == "k" else fresh.double()
            block = pools[x + "_pool"][pages]
            flat = block.flatten(0, 1)
            if op == "append8":
                scale = _exact_scales(pools[x + "_scale"][pages], raw, old, hi - lo,
                                      max(1.0, math.sqrt(2.0) * s["factor"]) if x == "k" else 1.0)
                if old:
                    ratio = (pools[x + "_scale"][pages[0]] / scale[0])[None, :, None]
                    flat[:old] = _e4m3(flat[:old] * ratio)
                of = torch.arange(old, old + n, device="cuda") // BLOCK
                fresh = _e4m3(fresh / scale[of][..., None])
                pools[x + "_scale"][pages] = scale
            flat[old:old + n] = fresh
            pools[x + "_pool"][pages] = flat.view(block.shape)
        a += n
    return {"q": q, **pools}


def _exact_scales(before, raw, old, blocks, grow):
    """Scales [blocks, Hkv] of the blocks whose slots from `old` on take the values raw."""
    rows = torch.zeros(blocks * BLOCK, *raw.shape[1:], dtype=torch.float64, device="cuda")
    rows[old:old + len(raw)] = raw.abs()
    top = rows.view(blocks, BLOCK, *raw.shape[1:]).amax((1, 3)) * grow
    # the smallest power of two with top <= 448 need; log2 may be one off at borders
    need = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=MIN_EXP))
    need = torch.where(need * E4M3_MAX < top, need * 2, need)
    need = torch.where((need / 2 * E4M3_MAX >= top) & (need > 2.0 ** MIN_EXP), need / 2, need)
    if old:
        need[0] = torch.maximum(need[0], before[0])
    return need


def _e4m3(x):
    """Nearest e4m3 value of each float64 value (ties to the even code)."""
    size = x.abs().clamp(max=E4M3_MAX)
    exp = torch.floor(torch.log2(size.clamp(min=2.0 ** -6)))
    step = torch.exp2(exp - 3)
    return torch.copysign((torch.round(size / step) * step).clamp(max=E4M3_MAX), x)


def _exact_prefix(s, case):
    ctx = _lens(case)[0]
    B, H, d = s["q"].shape
    Hkv = case["Hkv"]
    # about 1e12 products in 64 bits a second and less, and the gathers
    if 4 * d * H * sum(ctx) > 6e12:
        return None
    out = torch.zeros(B, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, c in enumerate(ctx):
        if not c:
            continue
        pages = s["table"][b, : (c + BLOCK - 1) // BLOCK].long()
        k, v = (s[x][pages].flatten(0, 1)[:c].double().transpose(0, 1) for x in ("k_pool", "v_pool"))
        q = s["q"][b].double().view(Hkv, H // Hkv, d)
        x = q @ k.transpose(1, 2) / math.sqrt(d)
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = (torch.softmax(x, -1) @ v).reshape(H, d)
    return {"out": out, "lse": lse}
