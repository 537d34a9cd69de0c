"""Rotary positions on the GPU: queries, keys and their gradients, and the
writes into the bf16 and the 8-bit cache that rotate on the way, against
64-bit arithmetic."""
import math

import numpy as np
import pytest

import cache_reference as cr
import rope_reference as rr
from exact_attention_33_gb300 import workloads as W
from gpu_helpers import assert_device_clean, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa_mod
    fa_mod.fa_device_status(clear=True)
    return fa_mod


def dev(a):
    return torch_mod().from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    return dev(np.asarray(a, dtype=np.float32)).to(torch_mod().bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def values(rng, *shape):
    """bf16 values of many magnitudes, float32."""
    mag = np.exp2(rng.integers(-6, 7, (*shape[:-1], 1))).astype(np.float32)
    return cr.bf16(rng, *shape) * mag


# ------------------------------------------------------------------ rows to rows

ROPE = [  # tokens or (B, N), H, Hkv, d, rot, interleaved, factor
    ((1,), 1, 1, 64, 64, False, 1.0),
    ((1,), 5, 0, 128, 128, True, 1.0),       # queries alone
    ((37,), 7, 1, 64, 16, False, 1.3),
    ((37,), 3, 3, 64, 48, True, 0.7),
    ((300,), 8, 2, 128, 112, False, 1.0),
    ((2, 513), 16, 4, 128, 128, False, 1.21),
    ((3, 1), 2, 2, 64, 32, True, 1.0),
    ((5000,), 32, 8, 128, 64, True, 1.0),
    ((9000,), 4, 1, 64, 64, False, 1.0),
]


@pytest.mark.parametrize("lead,H,Hkv,d,rot,inter,factor", ROPE)
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_rope(fa, lead, H, Hkv, d, rot, inter, factor, back, given):
    rng = np.random.default_rng(H + d + rot)
    q = values(rng, *lead, H, d)
    k = values(rng, *lead, Hkv, d) if Hkv else None
    pos = np.broadcast_to(np.arange(lead[-1]), lead)
    if given:
        pos = rng.integers(0, 1 << 20, lead)
        pos.flat[0], pos.flat[-1] = (1 << 31) - 1, -(1 << 31)
        if pos.size > 3:
            pos.flat[1], pos.flat[2] = 0, -7
    freq = rr.frequencies(rot)
    f = np.float32(factor)
    call = fa.fa_rope_bwd if back else fa.fa_rope
    got = call(bf16(q), None if k is None else bf16(k), dev(freq),
               positions=dev(pos.astype(np.int32)) if given else None, factor=factor,
               interleaved=inter)
    assert_device_clean()
    assert (got[1] is None) == (k is None)
    for x, y, name in ((q, got[0], "q"), (k, got[1], "k")):
        if x is None:
            continue
        assert y.shape == x.shape and y.is_contiguous()
        want = rr.rotate(x, pos, freq, f, inter, back)
        rr.close_bf16(host(y), want, rr.slack(x, pos, freq, f, inter), name)
        assert np.array_equal(host(y)[..., rot:], x[..., rot:].astype(np.float64))


def test_rope_far_positions_and_odd_frequencies(fa):
    """Turns of more than one a position, backwards, none at all, and positions
    at which an angle of 32 bits would be off by whole radians."""
    rng = np.random.default_rng(5)
    freq = np.array([0.0, 7.0, -0.5, 1e-9, 1.0, 6.283185307179586, 100.0, 0.9999999])
    x = values(rng, 6, 2, 64)
    pos = np.array([0, 1, 123456789, 16777217, (1 << 31) - 1, -2000000000])
    for inter in (False, True):
        got, _ = fa.fa_rope(bf16(x), None, dev(freq), dev(pos.astype(np.int32)), interleaved=inter)
        want = rr.rotate(x, pos, freq, 1.0, inter)
        rr.close_bf16(host(got), want, rr.slack(x, pos, freq, 1.0, inter))
    assert_device_clean()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_views_and_in_place(fa, inter):
    """Views of a fused projection, outputs that are views of another buffer
    (rows between them left alone), and outputs that are the inputs."""
    torch = torch_mod()
    rng = np.random.default_rng(6)
    H, Hkv, d, rot, T = 6, 2, 64, 32, 77
    fused = bf16(values(rng, T, H + 2 * Hkv, d))
    q, k = fused[:, :H], fused[:, H:H + Hkv]
    freq, pos = rr.frequencies(rot), np.arange(T)
    want = [rr.rotate(host(x), pos, freq, 1.0, inter) for x in (q, k)]
    off = [rr.slack(host(x), pos, freq, 1.0, inter) for x in (q, k)]
    box = torch.full((T, 2 * (H + Hkv), d), 3.0, dtype=torch.bfloat16, device="cuda")
    before = fused.clone()
    got = fa.fa_rope(q, k, dev(freq), interleaved=inter, q_out=box[:, :H], k_out=box[:, H + 1:H + 1 + Hkv])
    assert got[0].data_ptr() == box.data_ptr() and torch.equal(fused, before)
    for y, w, o in zip(got, want, off):
        rr.close_bf16(host(y), w, o)
    assert (box[:, H] == 3).all() and (box[:, H + 1 + Hkv:] == 3).all()
    fa.fa_rope(q, k, dev(freq), interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, box[:, :H]) and torch.equal(k, box[:, H + 1:H + 1 + Hkv])
    assert torch.equal(fused[:, H + Hkv:], before[:, H + Hkv:])
    assert_device_clean()


def test_rope_special_values(fa):
    """Infinities and NaN reach their own pair alone; zeros stay zeros."""
    d, rot = 64, 32
    x = np.zeros((3, 1, d), dtype=np.float32)
    x[0, 0, 3] = math.inf
    x[1, 0, 40] = math.nan       # passes through
    x[2, 0, 5] = math.nan
    freq = rr.frequencies(rot)
    got, _ = fa.fa_rope(bf16(x), None, dev(freq), dev(np.int32([4, 4, 4])))
    got = got.float().cpu().numpy()[:, 0]
    bad = ~np.isfinite(got)
    want = np.zeros_like(bad)
    want[0, [3, 3 + rot // 2]] = want[1, 40] = want[2, [5, 5 + rot // 2]] = True
    assert np.array_equal(bad, want) and (got[~bad] == 0).all()


def test_rope_gradient_is_the_transpose(fa):
    """<rope(x), g> and <x, rope_bwd(g)>, and differences of the rotation."""
    rng = np.random.default_rng(8)
    T, H, d, rot = 40, 3, 128, 96
    x, g, u = (values(rng, T, H, d) for _ in range(3))
    freq, pos = rr.frequencies(rot), rng.integers(0, 100000, T)
    at = dev(pos.astype(np.int32))
    y, _ = fa.fa_rope(bf16(x), None, dev(freq), at, factor=1.25)
    gx, _ = fa.fa_rope_bwd(bf16(g), None, dev(freq), at, factor=1.25)
    gx, y = host(gx), host(y)
    # each side's values are rounded once, plus fp32
    far = rr.U * (np.abs(y * g).sum() + np.abs(gx * x).sum()) * (1 + 2.0 ** -6)
    assert abs((y * g).sum() - (gx * x).sum()) <= far
    h = 1.0 / 64
    moved = [(rr.rotate(x.astype(float) + t * u, pos, freq, 1.25) * g).sum() for t in (h, -h)]
    diff = (moved[0] - moved[1]) / (2 * h)
    tol = (rr.U * np.abs(gx) + 2 * rr.slack(g, pos, freq, 1.25)) * np.abs(u)
    assert abs(diff - (gx * u).sum()) <= tol.sum() * (1 + 2.0 ** -6)


def test_rope_empty_and_refusals(fa):
    torch = torch_mod()
    f = dev(rr.frequencies(64))
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    a, b = fa.fa_rope(q, q, f)
    assert a.shape == b.shape == (0, 4, 64)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16, device="cuda")
    bad = [
        dict(q=q.float()), dict(q=q[..., ::2]), dict(q=q[:, :, :32]), dict(k=q[:2]),
        dict(inv_freq=f.float()), dict(inv_freq=f.cpu()), dict(inv_freq=torch.cat([f, f])),
        dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda")),
        dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
        dict(q_out=q[:, :2]), dict(k=None, k_out=q), dict(q=q.transpose(0, 1)),
        dict(q=q.expand(4, 4, 64)[:1].expand(4, 4, 64)),
    ]
    for more in bad:
        with pytest.raises(ValueError):
            fa.fa_rope(**{**dict(q=q, k=q, inv_freq=f), **more})
    for more in (dict(factor=0.0), dict(inv_freq=f[:12].contiguous())):
        with pytest.raises(fa.FaError):
            fa.fa_rope(**{**dict(q=q, k=q, inv_freq=f), **more})


def test_rope_stream_and_graph(fa):
    """On another stream than the current one, and captured and replayed on new inputs."""
    torch = torch_mod()
    rng = np.random.default_rng(9)
    freq = rr.frequencies(128)
    q, k = (torch.empty((64, h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pos, f = torch.zeros(64, dtype=torch.int32, device="cuda"), dev(freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.fa_rope(q, k, f, pos, q_out=qo, k_out=ko, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, k, f, pos, q_out=qo, k_out=ko)
    for turn in range(3):
        x, y, p = values(rng, 64, 8, 128), values(rng, 64, 2, 128), rng.integers(0, 5000, 64)
        q.copy_(bf16(x)), k.copy_(bf16(y)), pos.copy_(dev(p.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        for got, z in ((qo, x), (ko, y)):
            rr.close_bf16(host(got), rr.rotate(z, p, freq), rr.slack(z, p, freq), f"replay {turn}")


# ------------------------------------------------------------------ into a cache

APPEND = [  # context lengths, new tokens, H (0: none), Hkv, d, rot (0: none), interleaved, factor
    ([1], [1], 1, 1, 64, 64, False, 1.0),
    ([16, 17, 32], [16, 17, 16], 8, 2, 128, 128, False, 1.2),
    ([5, 40, 100, 16, 31], [1, 1, 1, 1, 1], 32, 8, 128, 128, False, 1.0),
    ([7, 90, 64], [0, 33, 1], 9, 3, 64, 16, True, 1.0),
    ([300, 1000], [257, 999], 7, 1, 64, 48, False, 0.6),
    ([50] * 40, [3] * 40, 2, 1, 128, 96, True, 1.0),
    ([130, 3], [100, 3], 0, 2, 128, 64, True, 1.0),        # no queries
    ([33, 70], [20, 70], 4, 2, 64, 0, False, 1.0),         # no rotation (bf16 cache)
]


def positions(ctx, new):
    return np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)]) if ctx else np.zeros(0)


class Run:
    """One write: inputs on both sides, and what has to come of it."""

    def __init__(self, ctx, new, H, Hkv, d, rot, inter, factor, seed, extra=0, width=None):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.ctx, self.new, self.inter, self.factor = ctx, new, inter, np.float32(factor)
        self.T = sum(new)
        self.q = values(rng, self.T + extra, H, d) if H else None
        self.k, self.v = (values(rng, self.T + extra, Hkv, d) for _ in "kv")
        self.freq = rr.frequencies(rot) if rot else np.zeros(0)
        self.pos = positions(ctx, new)
        self.table, self.blocks = cr.tables(ctx, seed, width=width)

    def slots(self):
        """Pool block and slot of each new token."""
        seq = np.repeat(np.arange(len(self.new)), self.new)
        return self.table[seq, self.pos // 16], self.pos % 16

    def call(self, fa, pools, fp8=False, **more):
        T = self.T
        name = "fa_cache_append_rope_fp8" if fp8 else "fa_cache_append_rope"
        q = None if self.q is None else bf16(self.q)
        kw = dict(factor=float(self.factor), interleaved=self.inter, **more)
        out = getattr(fa, name)(q, bf16(self.k), bf16(self.v),
                                dev(self.freq) if len(self.freq) else None, *pools, dev(self.table),
                                dev(np.int32(self.ctx)), dev(cu_of(self.new)), max(max(self.new), 1),
                                **kw)
        if q is not None and T:
            q64 = self.q[:T].astype(np.float64)
            rr.close_bf16(host(out)[:T], rr.rotate(q64, self.pos, self.freq, self.factor, self.inter),
                          rr.slack(q64, self.pos, self.freq, self.factor, self.inter, 9 if fp8 else 1),
                          "q")
        assert (out is None) == (q is None)
        return out


@pytest.mark.parametrize("ctx,new,H,Hkv,d,rot,inter,factor", APPEND)
def test_append(fa, ctx, new, H, Hkv, d, rot, inter, factor):
    torch = torch_mod()
    r = Run(ctx, new, H, Hkv, d, rot, inter, factor, seed=sum(ctx) + d, extra=5)
    pools = [bf16(r.rng.standard_normal((r.blocks, 16, Hkv, d))) for _ in "kv"]
    before = [p.clone() for p in pools]
    box = torch.full((r.T + 5, max(H, 1), d), 3.0, dtype=torch.bfloat16, device="cuda")
    r.call(fa, pools, **(dict(q_out=box) if H else {}))
    assert_device_clean()
    assert (box[r.T:] == 3).all()        # rows behind the last sequence
    blk, slot = r.slots()
    k64 = r.k[:r.T].astype(np.float64)
    got = host(pools[0])[blk, slot]
    rr.close_bf16(got, rr.rotate(k64, r.pos, r.freq, r.factor, inter),
                  rr.slack(k64, r.pos, r.freq, r.factor, inter), "k")
    assert np.array_equal(host(pools[1])[blk, slot], r.v[:r.T].astype(np.float64))
    if not rot:
        assert np.array_equal(got, k64)
    # every other slot as it was
    for p, b in zip(pools, before):
        b[blk, slot] = p[blk, slot]
        assert torch.equal(p, b)


@pytest.mark.parametrize("ctx,new,H,Hkv,d,rot,inter,factor", [a for a in APPEND if a[5]])
def test_append_fp8(fa, ctx, new, H, Hkv, d, rot, inter, factor):
    """Scales bit for bit, values that pass through and V bit for bit, rotated
    keys within half a step of e4m3 of the 64-bit value."""
    torch = torch_mod()
    r = Run(ctx, new, H, Hkv, d, rot, inter, factor, seed=sum(ctx) + d, extra=5)
    rng, T = r.rng, r.T
    codes = [rng.integers(0, 256, (r.blocks, 16, Hkv, d)).astype(np.uint8) for _ in "kv"]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0x3A
    scales = [np.exp2(rng.integers(-9, 3, (r.blocks, Hkv))).astype(np.float32) for _ in "kv"]
    pools = [dev(x) for x in (*codes, *scales)]
    box = torch.full((T + 5, max(H, 1), d), 3.0, dtype=torch.bfloat16, device="cuda")
    r.call(fa, pools, fp8=True, **(dict(q_out=box) if H else {}))
    assert_device_clean()
    assert (box[T:] == 3).all()
    got_k, got_v, got_ks, got_vs = (p.cpu().numpy() for p in pools)
    # values: the write of unrotated rows
    cr.append(r.v, codes[1], scales[1], r.table, ctx, new)
    assert np.array_equal(got_v, codes[1]) and np.array_equal(got_vs, scales[1])
    # keys: scales from the values before the rotation, older codes at them
    k64 = r.k[:T].astype(np.float64)
    turned = rr.rotate(k64, r.pos, r.freq, r.factor, inter)
    off = rr.slack(k64, r.pos, r.freq, r.factor, inter, 9)
    grow = rr.grow_of(factor)
    a = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        first = c - n
        for blk in range(first // 16, (c + 15) // 16 if n else 0):
            phys = r.table[b][blk]
            s0, s1 = max(0, first - blk * 16), min(16, c - blk * 16)
            at = slice(a + blk * 16 + s0 - first, a + blk * 16 + s1 - first)
            for h in range(Hkv):
                s = rr.need_scale(np.abs(r.k[at, h]).max(), grow)
                old = scales[0][phys, h]
                if s0 and old >= s:
                    s = float(old)
                elif s0:
                    was = W.e4m3_decode(codes[0][phys, :s0, h]).astype(np.float32)
                    codes[0][phys, :s0, h] = cr.encode(was * np.float32(old / s))
                assert got_ks[phys, h] == s, (b, blk, h)
                real = W.e4m3_decode(got_k[phys, s0:s1, h]) * s
                want = turned[at, h]
                step = np.maximum(rr.HALF_E4M3 * np.abs(want), s * 2.0 ** -10)
                # (a value on the border of two steps may go either way: the wider one counts)
                assert (np.abs(real - want) <= step * (1 + 2.0 ** -20) + 2 * off[at, h]).all()
                tail = cr.encode(r.k[at, h][:, rot:] / np.float32(s))
                assert np.array_equal(got_k[phys, s0:s1, h][:, rot:], tail)
                codes[0][phys, s0:s1, h] = got_k[phys, s0:s1, h]
                scales[0][phys, h] = s
        a += n
    assert np.array_equal(got_k, codes[0]) and np.array_equal(got_ks, scales[0])


@pytest.mark.parametrize("inter,factor,d", [(False, 1.0, 128), (True, 1.2, 128), (False, 1.1, 64)])
def test_append_fp8_few_codes_are_beside_the_nearest(fa, inter, factor, d):
    """Four million keys, rotated in fp32: where the code is not that of the exact
    value, that lies as near the border between both as fp32 may be off.  cos and
    sin are off by 0.82 units in their last place (1.64 x 2^-24 of themselves) and
    the angle by 2^-32 turns (2^-29 rad), the factor, a product and the sum round
    once each: 4.7 x 2^-24 of |a cos| + |b sin| and 2^-29 (|a| + |b|).

    With factor 1 there are 1 to 2 in a million of them (codes lie 2^-3 to 2^-4
    apart): 12 at most here.  With 1.2, which is 6/5, borders m 2^k with m a
    multiple of 3 are what bf16 values 5 (m/3) 2^(k-1) become at small angles, so
    their number says nothing there.  Compared are e4m3's normal values whose two
    terms do not cancel to less than a sixth."""
    torch = torch_mod()
    n, Hkv, seqs = 1024, 8, 4 * 128 // d
    g = torch.Generator(device="cuda").manual_seed(31)
    k = torch.randn((seqs * n, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(seqs * n // 16, generator=g, device="cuda").to(torch.int32).view(seqs, -1)
    ctx = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * n
    pools = [torch.zeros(seqs * n // 16, 16, Hkv, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros(seqs * n // 16, Hkv, device="cuda") for _ in "kv"]
    freq = dev(rr.frequencies(d))
    fa.fa_cache_append_rope_fp8(None, k, k, freq, *pools, *scales, table, ctx, cu, n, factor=factor,
                                interleaved=inter)
    assert_device_clean()
    order = table.flatten().long()
    got = pools[0][order].view(torch.float8_e4m3fn).double().view(seqs * n, Hkv, d)
    scale = scales[0][order].double().repeat_interleave(16, 0)[..., None]
    x = k.double()
    angle = torch.arange(n, dtype=torch.float64, device="cuda").repeat(seqs)[:, None, None] * freq
    fac = float(np.float32(factor))
    c, s = angle.cos() * fac, angle.sin() * fac
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        join = lambda u, v: torch.stack([u, v], -1).flatten(-2)  # noqa: E731
    else:
        a, b = x[..., :d // 2], x[..., d // 2:]
        join = lambda u, v: torch.cat([u, v], -1)  # noqa: E731
    y = join(a * c - b * s, a * s + b * c) / scale
    terms = join((a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()) / scale
    q = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    want = torch.round(y / q) * q
    # (the 64-bit angle is off by 2^-43: what is that near a border is left out)
    clear = ((y / q).abs() % 1 - 0.5).abs() > 2.0 ** -36
    fair = (y.abs() >= 2.0 ** -6) & (y.abs() * 6 >= terms) & clear
    assert fair.double().mean() > 0.8
    far = (got != want) & fair
    off = 5 * 2.0 ** -24 * terms + 2.0 ** -28 * join(*[(a.abs() + b.abs()) * fac] * 2) / scale
    border = ((y / q).abs() % 1 - 0.5).abs() * q
    assert (border <= off)[far].all()
    if factor == 1.0:
        assert far.sum() <= 12
    assert ((got - want).abs()[far] <= q[far] * (1 + 2.0 ** -20)).all()


def test_append_fp8_extremes(fa):
    """Zeros, the smallest and largest bf16 values, infinities and NaN, amax at a
    border, and an older scale that is no power of two."""
    d, rot = 64, 64
    k = np.zeros((48, 1, d), dtype=np.float32)
    k[3, 0, 0] = 2.0 ** -133
    k[16, 0, 5] = 3.3895314e38
    k[32, 0, :4] = math.inf, math.nan, 2.0, -1.0
    freq = rr.frequencies(rot)
    table = np.int32([[2, 0, 1]])
    pools = [dev(np.zeros((3, 16, 1, d), np.uint8)) for _ in "kv"]
    scales = [dev(np.full((3, 1), 0.7, np.float32)) for _ in "kv"]
    fa.fa_cache_append_rope_fp8(None, bf16(k), bf16(k), dev(freq), *pools, *scales, dev(table),
                                dev(np.int32([48])), dev(np.int32([0, 48])), 48)
    ks = scales[0].cpu().numpy()[[2, 0, 1], 0]
    grow = rr.grow_of(1.0)
    assert ks.tolist() == [2.0 ** -100, rr.need_scale(np.float32(3.3895314e38), grow),
                           rr.need_scale(2.0, grow)]
    got = W.e4m3_decode(pools[0].cpu().numpy()[[2, 0, 1]]).reshape(48, d)
    assert np.isnan(got[32, [0, 1, 32, 33]]).all() or not np.isfinite(got[32, [1, 33]]).any()
    assert np.isfinite(np.delete(got[32], [0, 1, 32, 33])).all() and np.isfinite(got[:32]).all()
    big = got[16, [5, 37]] * float(ks[1])
    want = rr.rotate(k[16].astype(np.float64), 16, freq)[0, [5, 37]]
    assert (np.abs(big - want) <= rr.HALF_E4M3 * np.abs(want) * 1.001 + float(ks[1]) * 2.0 ** -10).all()
    # token by token onto an older scale that is no power of two
    one = np.float32([[[0.3] * d]])
    fa.fa_cache_append_rope_fp8(None, bf16(one), bf16(one), dev(freq), *pools,
                                dev(np.full((3, 1), 0.7, np.float32)), scales[1], dev(table),
                                dev(np.int32([6])), dev(np.int32([0, 1])), 1)
    got = W.e4m3_decode(pools[0].cpu().numpy()[2, 5, 0]) * np.float32(0.7)
    want = rr.rotate(np.float64(bf16(one).float().cpu().numpy()[0]), 5, freq)[0]
    assert (np.abs(got - want) <= rr.HALF_E4M3 * np.abs(want) * 1.001 + 0.7 * 2.0 ** -10).all()
    assert_device_clean()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_bad_data(fa, fp8):
    """Sequences with bad bounds or contexts are skipped, bad blocks' keys and
    values are; everything else is written."""
    torch = torch_mod()
    H, Hkv, d = 4, 2, 64
    rng = np.random.default_rng(3)
    T = 12
    q, k, v = (bf16(values(rng, T, h, d)) for h in (H, Hkv, Hkv))
    f = dev(rr.frequencies(d))

    def write(ctx, cu, table, most):
        if fp8:
            pools = [torch.zeros((4, 16, Hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
            pools += [torch.ones((4, Hkv), device="cuda") for _ in "kv"]
            call = fa.fa_cache_append_rope_fp8
        else:
            pools = [torch.zeros((4, 16, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
            call = fa.fa_cache_append_rope
        out = torch.full_like(q, 3.0)
        call(q, k, v, f, *pools, dev(np.int32(table)), dev(np.int32(ctx)), dev(np.int32(cu)), most,
             q_out=out)
        return out, [p.float().abs().sum((1, 2, 3)) > 0 for p in pools[:2]], fa.fa_device_status()

    good, used, st = write([4, 8], [0, 4, 12], [[0], [1]], 8)
    assert st == 0 and all(u.tolist() == [True, True, False, False] for u in used)
    assert not (good == 3).all((1, 2)).any()
    out, used, st = write([4, 8], [0, 4, 12], [[0], [4]], 8)     # a block outside the pool
    assert st == fa.FA_DEV_BAD_BLOCK and all(u.tolist() == [True, False, False, False] for u in used)
    assert torch.equal(out, good)                                # the queries have no block
    out, used, st = write([4, 7], [0, 4, 12], [[0], [1]], 8)     # more new tokens than context
    assert st == fa.FA_DEV_BAD_CTX and all(u.tolist() == [True, False, False, False] for u in used)
    assert torch.equal(out[:4], good[:4]) and (out[4:] == 3).all()
    out, used, st = write([4, 17], [0, 4, 12], [[0], [1]], 8)    # beyond the table
    assert st == fa.FA_DEV_BAD_CTX and (out[4:] == 3).all()
    out, used, st = write([4, 8], [0, 4, 12], [[0], [1]], 7)     # longer than max_new
    assert st == fa.FA_DEV_BAD_SEQLEN and (out[4:] == 3).all()
    out, used, st = write([4, 8], [0, 4, 13], [[0], [1]], 9)     # beyond the tokens
    assert st == fa.FA_DEV_BAD_SEQLEN and (out[4:] == 3).all()
    out, used, st = write([4, 8], [0, -1, 8], [[0], [1]], 9)
    assert st == fa.FA_DEV_BAD_SEQLEN and (out == 3).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_in_place_views(fa, fp8):
    """q, k and v as views of one projection, q rotated in its place."""
    torch = torch_mod()
    r = Run([20, 61], [9, 33], 6, 2, 64, 64, False, 1.0, seed=11)
    fused = torch.cat([bf16(x) for x in (r.q, r.k, r.v)], 1)
    q, k, v = fused[:, :6], fused[:, 6:8], fused[:, 8:]

    def pools():
        if fp8:
            return [torch.zeros((r.blocks, 16, 2, 64), dtype=torch.float8_e4m3fn, device="cuda")
                    for _ in "kv"] + [torch.ones((r.blocks, 2), device="cuda") for _ in "kv"]
        return [torch.zeros((r.blocks, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    call = fa.fa_cache_append_rope_fp8 if fp8 else fa.fa_cache_append_rope
    args = dev(r.table), dev(np.int32(r.ctx)), dev(cu_of(r.new)), 33
    a, b = pools(), pools()
    want = call(bf16(r.q), bf16(r.k), bf16(r.v), dev(r.freq), *a, *args)
    got = call(q, k, v, dev(r.freq), *b, *args, q_out=q)
    assert got.data_ptr() == fused.data_ptr() and torch.equal(q, want)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(k, bf16(r.k)) and torch.equal(v, bf16(r.v))
    assert_device_clean()


def test_append_far_offsets(fa):
    """A pool of more than 2^31 values: slots past the reach of 32-bit offsets."""
    torch = torch_mod()
    Hkv, d = 64, 128
    blocks = (1 << 31) // (16 * Hkv * d) + 8
    pools = [torch.zeros((blocks, 16, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    rng = np.random.default_rng(0)
    k, v = (values(rng, 3, Hkv, d) for _ in "kv")
    freq = rr.frequencies(d)
    fa.fa_cache_append_rope(None, bf16(k), bf16(v), dev(freq), *pools, dev(np.int32([[blocks - 1]])),
                            dev(np.int32([7])), dev(np.int32([0, 3])), 3)
    rr.close_bf16(host(pools[0][-1, 4:7]), rr.rotate(k, np.arange(4, 7), freq),
                  rr.slack(k, np.arange(4, 7), freq))
    assert np.array_equal(host(pools[1][-1, 4:7]), v.astype(np.float64))
    assert not pools[0][:-1].any() and not pools[1][-1, 7:].any()
    assert_device_clean()


def _rows_of(table, pool, b, c, scale=None):
    blocks = table[b, : (c + 15) // 16]
    x = pool[dev(blocks.astype(np.int64))].double()
    if scale is not None:
        x = x * scale[dev(blocks.astype(np.int64))].double()[:, None, :, None]
    return x.flatten(0, 1)[:c]


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_run(fa, fp8):
    """Prompts, then tokens one by one: each step writes the cache, rotates its
    queries and attends; against attention in 64 bits over what was written, and
    the written keys against rotated ones."""
    torch = torch_mod()
    rng = np.random.default_rng(12)
    H, Hkv, d, rot = 8, 2, 128, 128
    lens, steps = [70, 1, 33], 3
    final = [n + steps for n in lens]
    table, blocks = cr.tables(final, 5)
    dtable, f = dev(table), dev(rr.frequencies(rot))
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pools = [torch.zeros((blocks, 16, Hkv, d), dtype=kind, device="cuda") for _ in "kv"]
    scales = [torch.ones((blocks, Hkv), device="cuda") for _ in "kv"] if fp8 else []
    raw = [[] for _ in lens]   # every key as it was projected
    for step in range(steps + 1):
        new = lens if step == 0 else [1] * len(lens)
        ctx = [n + step for n in lens]
        q, k, v = (cr.bf16(rng, sum(new), h, d) for h in (H, Hkv, Hkv))
        for b, part in enumerate(np.split(k, cu_of(new)[1:-1])):
            raw[b].append(part)
        dctx, cu = dev(np.int32(ctx)), dev(cu_of(new))
        name = "fa_cache_append_rope_fp8" if fp8 else "fa_cache_append_rope"
        qr = getattr(fa, name)(bf16(q), bf16(k), bf16(v), f, *pools, *scales, dtable, dctx, cu, max(new))
        if step == 0:
            call = fa.fa_fwd_paged_fp8 if fp8 else fa.fa_fwd_paged
            out, _ = call(qr, *pools, *scales, dtable, dctx, cu, max(new), max(ctx))
        else:
            call = fa.fa_decode_paged_fp8 if fp8 else fa.fa_decode_paged
            out, _ = call(qr, *pools, *scales, dtable, dctx, max(ctx))
        a = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            kk = _rows_of(table, pools[0], b, c, scales[0] if fp8 else None)
            vv = _rows_of(table, pools[1], b, c, scales[1] if fp8 else None)
            for h in range(H):
                x = qr[a:a + n, h].double() @ kk[:, h // (H // Hkv)].T / math.sqrt(d)
                hide = torch.arange(c, device="cuda") > torch.arange(c - n, c, device="cuda")[:, None]
                p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                w = vv[:, h // (H // Hkv)]
                # a weight is rounded once (2^-8 of itself at most), V over the 8-bit
                # cache exactly, the output once; scores and sums are fp32
                size = p @ w.abs()
                tol = 2.0 ** -8 * size + 2.0 ** -8 * (p @ w).abs() + 2.0 ** -12 * size
                assert ((out[a:a + n, h].double() - p @ w).abs() <= tol).all(), (step, b, h)
            a += n
    assert_device_clean()
    for b, c in enumerate(final):
        want = rr.rotate(np.concatenate(raw[b]), np.arange(c), rr.frequencies(rot))
        got = _rows_of(table, pools[0], b, c, scales[0] if fp8 else None).cpu().numpy()
        # bf16: one rounding; e4m3: half a step, and half a finer one for each growth of a
        # block's scale (below e4m3's normal range)
        tol = np.maximum((2.0 ** -4 if fp8 else 2.0 ** -8) * np.abs(want), 2.0 ** -8 if fp8 else 1e-6)
        assert (np.abs(got - want) <= tol * 1.01 + 1e-5).all()


def test_training_run(fa):
    """Rotation, attention and both gradients against differences of the whole
    in 64 bits."""
    torch = torch_mod()
    rng = np.random.default_rng(13)
    B, N, H, Hkv, d, rot = 2, 50, 4, 2, 64, 32
    q, k, v, g = (cr.bf16(rng, B, N, h, d) for h in (H, Hkv, Hkv, H))
    f = dev(rr.frequencies(rot))
    qr, kr = fa.fa_rope(bf16(q), bf16(k), f)
    out, lse = fa.fa_fwd(qr, kr, bf16(v), causal=True)
    dq, dk, dv = fa.fa_bwd(qr, kr, bf16(v), out, lse, bf16(g), causal=True)
    dq, dk = fa.fa_rope_bwd(dq, dk, f)
    assert_device_clean()
    freq, pos = rr.frequencies(rot), np.arange(N)

    def loss(q, k, v):
        q, k = (torch.from_numpy(rr.rotate(x, pos, freq)) for x in (q, k))
        k, v = (x.repeat_interleave(H // Hkv, 2) for x in (k, torch.from_numpy(np.asarray(v, float))))
        x = torch.einsum("bnhd,bmhd->bhnm", q, k) / math.sqrt(d)
        x = x.masked_fill(torch.ones(N, N).triu(1).bool(), -math.inf)
        o = torch.einsum("bhnm,bmhd->bnhd", torch.softmax(x, -1), v)
        return float((o * torch.from_numpy(np.asarray(g, float))).sum())
    args = [np.asarray(x, float) for x in (q, k, v)]
    for i, grad in enumerate((dq, dk, dv)):
        grad = host(grad)
        for _ in range(3):
            u = rng.standard_normal(args[i].shape)
            h = 1e-5
            sides = [loss(*(x + s * h * u if j == i else x for j, x in enumerate(args))) for s in (1, -1)]
            diff = (sides[0] - sides[1]) / (2 * h)
            # the library's gradients are within 1.5e-2 relative RMS of the formula's
            # (its own tests); against a random direction that is 1.5e-2 |grad| and one
            # rounding more, times a normal factor (5 of them: one in a million)
            assert abs(diff - (grad * u).sum()) <= 5 * 2e-2 * np.linalg.norm(grad), i


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_hold_their_last_places(fa, inter, back, sign):
    """a cos t - b sin t with b t next to a, so that what sin is off by shows: angles
    from 2^-28 to a quarter, both signs.

    From 2^-32 of a turn up sin is within 3.1 x 2^-24 of itself and cos within 0.98;
    b sin t and a cos t are about 1, and their products round once each (2^-24 and
    2^-25; the sum's rounding is of the small result); turns a position are held to
    2^-64, at most 2^-26 of the angles here: 5.9 x 2^-24 in all, and half a step of
    bf16."""
    rng = np.random.default_rng(5)
    rot, heads = 128, 3
    for pos, least in [(1, -27), (7, -27), (-1, -27), (-12, -20), (100003, -14)] * 5:
        mag = np.exp2(rng.uniform(least, -2, rot // 2))
        b = np.exp2(np.round(-np.log2(mag))) * np.round(rng.uniform(1, 2, rot // 2) * 128) / 128 * sign
        freq = (1 - 2.0 ** -13) / b / pos
        x = rr.join(np.ones((1, heads, rot // 2)),
                    np.broadcast_to(-b if back else b, (1, heads, rot // 2)),
                    np.zeros((1, heads, rot)), rot, inter)
        call = fa.fa_rope_bwd if back else fa.fa_rope
        out, _ = call(bf16(x), None, dev(freq), positions=dev(np.int32([pos])), interleaved=inter)
        got, _ = rr.split(host(out), rot, inter)
        t = freq * float(pos)
        want = np.cos(t) - b * np.sin(t)
        off = np.abs(got[0] - want) - (rr.U * np.abs(want) + (1 + rr.U) * 5.9 * 2.0 ** -24)
        assert off.max() <= 0, (pos, t[off.max(0).argmax()], off.max())
    assert_device_clean()


def test_slow_pairs_at_small_positions(fa):
    """The slowest pair of a stretched context at its first positions: sin is as
    near as bf16 lets it be."""
    freq = rr.frequencies(128, base=500000.0) / 32
    pos = np.arange(-5, 6, dtype=np.int32)
    x = np.zeros((len(pos), 1, 128))
    x[..., :64] = 1.0
    out, _ = fa.fa_rope(bf16(x), None, dev(freq), positions=dev(pos))
    got = host(out)[:, 0, 64:]
    want = np.sin(pos[:, None] * freq)
    assert (np.abs(got - want) <= (rr.U + 4 * 2.0 ** -24) * np.abs(want)).all()


@pytest.mark.parametrize("ctx,new,H,Hkv,d,rot,inter,factor", [a for a in APPEND if a[5]])
def test_both_writes_turn_alike(fa, ctx, new, H, Hkv, d, rot, inter, factor):
    """The 8-bit write's queries are the bf16 write's bit for bit, and its keys
    within half a step of e4m3 and what fp32 may be off by.

    cos and sin are within 2.5 x 2^-24 of themselves (3.1 for the smallest angles),
    the factor, the products and the sum round once each: 6.1 x 2^-24 of |a cos| + |b
    sin|; the product of position and frequency is held to 2^-53 of itself here and
    there, so the angle to 2^-51 (and 2^-50 rad).  Half a step at the value that was rounded is that
    at the exact one and 2^-4 of what lies between."""
    torch = torch_mod()
    r = Run(ctx, new, H, Hkv, d, rot, inter, factor, seed=sum(ctx) + d)
    pools = [torch.zeros((r.blocks, 16, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pools8 = [torch.zeros((r.blocks, 16, Hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros((r.blocks, Hkv), device="cuda") for _ in "kv"]
    q = r.call(fa, pools)
    q8 = r.call(fa, [*pools8, *scales], fp8=True)
    assert_device_clean()
    assert q is None or torch.equal(q.view(torch.int16), q8.view(torch.int16))
    blk, slot = r.slots()
    s = scales[0].double().cpu().numpy()[blk][..., None]
    real = W.e4m3_decode(pools8[0].cpu().numpy()[blk, slot]) * s
    k64 = r.k[:r.T].astype(np.float64)
    want = rr.rotate(k64, r.pos, r.freq, r.factor, inter)
    t = np.asarray(r.pos, np.float64)[:, None, None] * r.freq
    a, b = (np.abs(z) for z in rr.split(k64, rot, inter))
    c, sn = np.abs(np.cos(t)), np.abs(np.sin(t))
    turn = (np.abs(t) * 2.0 ** -51 + 2.0 ** -50) * (a + b)
    off = float(r.factor) * rr.join(a * c + b * sn, a * sn + b * c, np.zeros_like(k64), rot, inter)
    off = 6.1 * 2.0 ** -24 * off + float(r.factor) * rr.join(turn, turn, np.zeros_like(k64), rot, inter)
    tol = np.maximum(rr.HALF_E4M3 * (np.abs(want) + off), s * 2.0 ** -10) + off
    assert (np.abs(real - want) <= tol * (1 + 2.0 ** -40)).all()
