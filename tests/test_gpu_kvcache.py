"""The 8-bit paged cache: the quantising write (bit for bit), attention over
it for single tokens against 64-bit arithmetic, and a serving run of both."""
import math

import numpy as np
import pytest

import cache_reference as cr
import window_reference as ref
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


def dev(a, dtype=None):
    torch = torch_mod()
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(a):
    return dev(a, torch_mod().bfloat16)


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Cache:
    """A cache on the device beside its NumPy twin."""

    def __init__(self, ctx, Hkv, d, seed, width=None):
        rng = np.random.default_rng(seed)
        self.table, blocks = cr.tables(ctx, seed, width=width)
        self.pool, self.scale = {}, {}
        for x in "kv":
            # every finite code, so also those of stale slots
            codes = rng.integers(0, 256, (blocks, 16, Hkv, d)).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x3A
            self.pool[x] = codes
            self.scale[x] = np.exp2(rng.integers(-9, -4, (blocks, Hkv))).astype(np.float32)
        self.dpool = {x: dev(self.pool[x]) for x in "kv"}
        self.dscale = {x: dev(self.scale[x]) for x in "kv"}
        self.dtable = dev(self.table)

    def args(self):
        return self.dpool["k"], self.dpool["v"], self.dscale["k"], self.dscale["v"], self.dtable

    def append(self, fa, k, v, ctx, new, **more):
        for x, t in (("k", k), ("v", v)):
            cr.append(t, self.pool[x], self.scale[x], self.table, ctx, new)
        kd, vd = more.pop("tensors", None) or (bf16(k), bf16(v))
        fa.fa_cache_append_fp8(kd, vd, *self.args(), dev(np.int32(ctx)), dev(cu_of(new)),
                               max(max(new), 1), **more)

    def check(self, what=""):
        for x in "kv":
            assert np.array_equal(self.dscale[x].cpu().numpy(), self.scale[x]), f"{what} {x} scale"
            got = self.dpool[x].cpu().numpy()
            nan = (got & 0x7F) == 0x7F
            assert np.array_equal(nan, (self.pool[x] & 0x7F) == 0x7F), f"{what} {x} NaN"
            assert np.array_equal(got[~nan], self.pool[x][~nan]), f"{what} {x} codes"

    def rows(self, x, b, ctx):
        """Keys or values of sequence b in 64 bits, [ctx, Hkv, d], on the device."""
        blocks = self.table[b, : (ctx + 15) // 16]
        return dev(cr.real(self.pool[x][blocks], self.scale[x][blocks]).reshape(
            -1, *self.pool[x].shape[2:])[:ctx])


# ------------------------------------------------------------------ the write

APPEND = [
    ([1], [1], 1, 64),
    ([16, 17, 32], [16, 17, 16], 2, 128),
    ([5, 40, 100, 16, 31], [1, 1, 1, 1, 1], 8, 128),    # single tokens, one begins a block
    ([7, 90, 64], [0, 33, 1], 3, 64),                     # a sequence without new tokens
    ([300, 1000], [257, 999], 2, 64),
    ([50] * 40, [3] * 40, 1, 128),
]


@pytest.mark.parametrize("ctx,new,Hkv,d", APPEND)
def test_append(fa, ctx, new, Hkv, d):
    rng = np.random.default_rng(len(ctx) + d)
    c = Cache(ctx, Hkv, d, seed=sum(ctx))
    t = sum(new)
    # magnitudes from far below to far above what the blocks hold
    mag = np.exp2(rng.integers(-12, 9, (t, Hkv, 1))).astype(np.float32)
    c.append(fa, cr.bf16(rng, t, Hkv, d) * mag, cr.bf16(rng, t, Hkv, d), ctx, new)
    assert_device_clean()
    c.check()


def test_append_extremes(fa):
    """Zeros, bf16's smallest and largest values, infinities and NaN, and
    amax at the border of a power of two."""
    Hkv, d = 2, 64
    rows = np.zeros((48, Hkv, d), dtype=np.float32)
    rows[1, 0, 0] = 2.0 ** -133          # subnormal: a scale of 2^-100
    rows[16, 0, :4] = 448, -448, 0.1, 3e-3
    rows[16, 1, :4] = 450, 1, -0.5, 1e-5  # just above the border
    rows[32, 0, :5] = math.inf, -math.inf, math.nan, 7.0, -3.0
    rows[33, 1, :2] = 3.3895314e38, 1e30
    c = Cache([48], Hkv, d, seed=1)
    c.append(fa, rows, -rows, [48], [48])
    assert_device_clean()
    c.check()
    assert c.scale["k"][c.table[0, 0]].tolist() == [2.0 ** -100] * 2
    assert c.scale["k"][c.table[0, 1]].tolist() == [1.0, 2.0]
    assert c.scale["k"][c.table[0, 2], 0] == 2.0 ** -6


def test_append_token_by_token(fa):
    """A block filled one token at a time, its scale growing on the way, and
    an older scale that is no power of two."""
    rng = np.random.default_rng(3)
    Hkv, d = 3, 128
    c = Cache([40], Hkv, d, seed=4)
    c.append(fa, *(cr.bf16(rng, 5, Hkv, d) for _ in "kv"), [5], [5])
    for x in "kv":  # as another writer might have left it
        c.scale[x][c.table[0, 0]] = np.float32([0.0037, 0.02, 3.0])
        c.dscale[x].copy_(dev(c.scale[x]))
    for n in range(6, 41):
        grow = np.float32(2.0 ** ((n % 7) * 2 - 6))
        c.append(fa, *(cr.bf16(rng, 1, Hkv, d) * grow for _ in "kv"), [n], [1])
        c.check(f"token {n}")
    assert_device_clean()


def test_append_from_a_fused_projection(fa):
    """k and v as views of one [T, (H + 2 Hkv) d] tensor."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    H, Hkv, d, ctx = 4, 2, 64, [30, 77]
    qkv = cr.bf16(rng, sum(ctx), H + 2 * Hkv, d)
    t = bf16(qkv)
    c = Cache(ctx, Hkv, d, seed=6)
    c.append(fa, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], ctx, ctx,
             tensors=(t[:, H:H + Hkv], t[:, H + Hkv:]))
    assert_device_clean()
    c.check()


def test_append_reports_bad_arguments_of_the_device(fa):
    """A bad context length, a bad block id and a bad offset each skip what
    they concern; the sequences beside them are written."""
    torch = torch_mod()
    rng = np.random.default_rng(7)
    Hkv, d, ctx, new = 2, 64, [20, 33, 18, 40], [20, 3, 2, 8]
    c = Cache(ctx, Hkv, d, seed=8)
    k, v = (cr.bf16(rng, sum(new), Hkv, d) for _ in "kv")
    good, bad = [1], {0: "block", 2: "ctx"}
    bad_table = c.table.copy()
    bad_table[0, 1] = 10 ** 6
    lens, cu = np.int32(ctx), cu_of(new)
    lens[2] = 1                       # fewer than its new tokens
    want = c.table[0, 0]
    # the twin: sequence 0's first block, sequence 1 and sequence 3
    for x, t in (("k", k), ("v", v)):
        cr.append(t[:16], c.pool[x], c.scale[x], c.table[:1], [16], [16])
        cr.append(t[20:23], c.pool[x], c.scale[x], c.table[1:2], [33], [3])
        cr.append(t[25:], c.pool[x], c.scale[x], c.table[3:], [40], [8])
    fa.fa_cache_append_fp8(bf16(k), bf16(v), *c.args()[:4], dev(bad_table), dev(lens), dev(cu), 20)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_BLOCK | fa.FA_DEV_BAD_CTX
    c.check()
    # more new tokens than max_new says: reported, nothing of it written
    fa.fa_cache_append_fp8(bf16(-k), bf16(v), *c.args(), dev(np.int32(ctx)), dev(cu), 2)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_SEQLEN
    cr.append(-k[23:25], c.pool["k"], c.scale["k"], c.table[2:3], [18], [2])
    cr.append(v[23:25], c.pool["v"], c.scale["v"], c.table[2:3], [18], [2])
    c.check("max_new")


# ------------------------------------------------------------------ single tokens

def check_decode(out, lse, q, c, ctx, window, sinks, what):
    H, Hkv = q.shape[1], c.pool["k"].shape[2]
    for b, n in enumerate(ctx):
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        for h in range(H):
            kv = h // (H // Hkv)
            o, l, tol = cr.decode_rows(q[b:b + 1, h].double(), k[:, kv], v[:, kv], window, sinks)
            ref.assert_within(out[b:b + 1, h], o, tol, f"{what} seq {b} head {h}")
            ref.assert_lse(lse[b:b + 1, h], l, f"{what} seq {b} head {h}")


DECODE = [
    ([1], 1, 1, 64, 0, 0),
    ([5, 16, 17, 0, 300], 4, 2, 128, 0, 0),
    ([700, 33, 1024], 8, 1, 64, 0, 0),
    ([1000, 999, 31, 32], 6, 2, 128, 0, 0),
    ([2000, 1], 32, 2, 128, 0, 0),               # group of 16
    ([47, 48, 49], 9, 1, 64, 0, 0),
    ([3000], 7, 1, 128, 0, 0),
    ([700, 33, 1024], 8, 1, 64, 100, 20),
    ([640, 641, 655, 656], 2, 2, 64, 64, 16),
    ([1000, 40], 4, 2, 128, 1, 0),
    ([5000, 130], 16, 2, 128, 4096, 64),
    ([300, 40], 3, 1, 64, 10000, 2),
]


@pytest.mark.parametrize("ctx,H,Hkv,d,window,sinks", DECODE)
def test_decode(fa, ctx, H, Hkv, d, window, sinks):
    """Stale and hidden slots hold NaN codes; blocks without a visible key
    have no table entry."""
    torch = torch_mod()
    c = Cache(ctx, Hkv, d, seed=20 + d)
    table = c.table.copy()
    for b, n in enumerate(ctx):
        for blk in range((n + 15) // 16):
            hidden = [t for t in range(blk * 16, blk * 16 + 16)
                      if t >= n or (window and t < n - window and t >= sinks)]
            for x in "kv":
                c.dpool[x][int(c.table[b, blk]), [t % 16 for t in hidden]] = 0x7F
            if len(hidden) == 16:
                table[b, blk] = -5
    q = bf16(cr.bf16(np.random.default_rng(d), len(ctx), H, d))
    out, lse = fa.fa_decode_paged_fp8(q, *c.args()[:4], dev(table), dev(np.int32(ctx)), max(ctx),
                                      window, sinks)
    assert_device_clean()
    check_decode(out, lse, q, c, ctx, window, sinks, "decode")


def test_decode_scales_far_apart(fa):
    """Scales over fifty powers of two, zeros, and queries of any size: the
    block that matters may be the one with the smallest scale."""
    ctx, H, Hkv, d = [200, 96], 4, 2, 64
    rng = np.random.default_rng(30)
    for case in range(4):
        c = Cache(ctx, Hkv, d, seed=31 + case)
        blocks = c.pool["k"].shape[0]
        if case == 0:
            c.scale["v"][:] = np.exp2(rng.integers(-40, 10, (blocks, Hkv)))
        elif case == 1:  # the heavy keys' values are small
            c.scale["k"][:] = np.exp2(rng.integers(-12, -3, (blocks, Hkv)))
            c.scale["v"][:] = 2.0 ** -20 / c.scale["k"] ** 3
        elif case == 2:
            c.scale["v"][::2] = 0.0
            c.scale["k"][:] = 0.013 * rng.random((blocks, Hkv))
        for x in "kv":
            c.scale[x] = c.scale[x].astype(np.float32)
            c.dscale[x].copy_(dev(c.scale[x]))
        q = cr.bf16(rng, 2, H, d)
        if case == 3:
            q = q * np.float32([[[1e-30], [2.0 ** -120], [0.0], [100.0]]])
        q = bf16(q)
        out, lse = fa.fa_decode_paged_fp8(q, *c.args(), dev(np.int32(ctx)), 200)
        assert_device_clean()
        check_decode(out, lse, q, c, ctx, 0, 0, f"case {case}")


def test_decode_reports_and_recovers(fa):
    torch = torch_mod()
    ctx, H, Hkv, d = [100, 200, 64], 4, 2, 128
    c = Cache(ctx, Hkv, d, seed=40)
    table, lens = c.table.copy(), np.int32(ctx)
    table[0, 6], lens[2] = c.pool["k"].shape[0], -1
    q = bf16(cr.bf16(np.random.default_rng(41), 3, H, d))
    ws = fa.new_workspace(fa.fa_decode_window_workspace_size(3, H, Hkv, d, 200, 0, 0))
    out, lse = fa.fa_decode_paged_fp8(q, *c.args()[:4], dev(table), dev(lens), 200, workspace=ws)
    torch.cuda.synchronize()
    bits = fa.FA_DEV_BAD_BLOCK | fa.FA_DEV_BAD_CTX
    assert fa.fa_last_device_status(ws) == bits and fa.fa_device_status(clear=True) == bits
    check_decode(out[1:2], lse[1:2], q[1:2], _Only(c, 1), [200], 0, 0, "beside")
    out, lse = fa.fa_decode_paged_fp8(q, *c.args(), dev(np.int32(ctx)), 200, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status(ws) == 0
    check_decode(out, lse, q, c, ctx, 0, 0, "after")


class _Only:
    """One sequence of a cache."""

    def __init__(self, c, b):
        self.pool, self.rows = c.pool, lambda x, _, n: c.rows(x, b, n)


# ------------------------------------------------------------------ chunks

CHUNKS = [
    ([1], [1], 1, 1, 64, 0, 0),
    ([5, 200], [5, 129], 2, 1, 64, 0, 0),
    ([300, 129, 40], [100, 129, 1], 4, 2, 128, 0, 0),
    ([700, 16, 0], [300, 3, 2], 3, 1, 64, 0, 0),      # row pairs; no context at all
    ([1000, 30], [260, 40], 6, 2, 128, 0, 0),         # a chunk longer than its context
    ([2050], [17], 16, 1, 128, 0, 0),
    ([900, 41], [400, 20], 3, 1, 128, 128, 0),        # row pairs with a window
    ([1500, 77], [256, 77], 4, 1, 64, 200, 140),
    ([2000, 15], [300, 15], 8, 2, 128, 500, 4),
    ([640], [384], 5, 5, 128, 1, 0),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,d,window,sinks", CHUNKS)
def test_chunks(fa, ctx, new, H, Hkv, d, window, sinks):
    """Stale slots hold NaN codes; blocks behind the first query's window have
    no table entry."""
    c = Cache(ctx, Hkv, d, seed=80 + d)
    table = c.table.copy()
    for b, (n, m) in enumerate(zip(ctx, new)):
        if n % 16:
            for x in "kv":
                c.dpool[x][int(c.table[b, n // 16]), n % 16:] = 0x7F
        for blk in range((n + 15) // 16):
            if window and blk * 16 >= sinks and blk * 16 + 16 <= n - m + 1 - window:
                table[b, blk] = 1 << 29
    cu = cu_of(new)
    q = bf16(cr.bf16(np.random.default_rng(d), cu[-1], H, d))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args()[:4], dev(table), dev(np.int32(ctx)), dev(cu),
                                   max(new), max(ctx), window, sinks)
    assert_device_clean()
    check_chunks(out, lse, q, c, ctx, cu, window, sinks)


def check_chunks(out, lse, q, c, ctx, cu, window, sinks, rounded=False):
    torch = torch_mod()
    H, Hkv = q.shape[1], c.pool["k"].shape[2]
    for b, n in enumerate(ctx):
        a, e = int(cu[b]), int(cu[b + 1])
        if a == e:
            continue
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        if rounded:
            v = v.to(torch.bfloat16).double()
        for h in range(H):
            kv = h // (H // Hkv)
            o, l, tol = ref.forward(q[a:e, h].double(), k[:, kv], v[:, kv], window, sinks)
            ref.assert_within(out[a:e, h], o, tol, f"seq {b} head {h}")
            ref.assert_lse(lse[h, a:e], l, f"seq {b} head {h}")


@pytest.mark.parametrize("batch", [1, 32, 33])
def test_chunks_of_many_sequences(fa, batch):
    """Each sequence gets its own rows whatever order the sequences start in:
    ascending, equal and empty contexts, up to and past a warp's 32."""
    H, Hkv, d = 2, 1, 64
    ctx = [40] if batch == 1 else [(7 * b) // 3 * 5 for b in range(batch)]
    new = [min(n, 1 + b % 4) for b, n in enumerate(ctx)]
    c = Cache(ctx, Hkv, d, seed=95 + batch)
    cu = cu_of(new)
    q = bf16(cr.bf16(np.random.default_rng(batch), cu[-1], H, d))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), dev(np.int32(ctx)), dev(cu), max(new), max(ctx))
    assert_device_clean()
    check_chunks(out, lse, q, c, ctx, cu, 0, 0)


def test_chunks_with_any_scale(fa):
    """Scales that are no powers of two: V rounded to bf16 once."""
    torch = torch_mod()
    ctx, new, H, Hkv, d = [333, 90], [140, 90], 4, 2, 128
    c = Cache(ctx, Hkv, d, seed=90)
    rng = np.random.default_rng(91)
    for x in "kv":
        c.scale[x] = (0.002 + 0.01 * rng.random(c.scale[x].shape)).astype(np.float32)
        c.dscale[x].copy_(dev(c.scale[x]))
    cu = cu_of(new)
    q = bf16(cr.bf16(rng, cu[-1], H, d))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), dev(np.int32(ctx)), dev(cu), max(new), max(ctx))
    assert_device_clean()
    check_chunks(out, lse, q, c, ctx, cu, 0, 0, rounded=True)


def test_chunks_report_bad_blocks(fa):
    torch = torch_mod()
    ctx, new, H, Hkv, d = [200, 100], [50, 20], 4, 2, 64
    c = Cache(ctx, Hkv, d, seed=92)
    table, lens = c.table.copy(), np.int32(ctx)
    table[0, 3] = -1
    cu = cu_of(new)
    q = bf16(cr.bf16(np.random.default_rng(93), cu[-1], H, d))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args()[:4], dev(table), dev(lens), dev(cu), 50, 200)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_BLOCK
    check_chunks(out[50:], lse[:, 50:], q[50:], _Only(c, 1), [100], [0, 20], 0, 0)
    lens[1] = 10 ** 6
    fa.fa_fwd_paged_fp8(q, *c.args(), dev(lens), dev(cu), 50, 200)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_CTX


# ------------------------------------------------------------------ together

def test_serving_run(fa):
    """Prompts written into the cache, then tokens one by one: write, attend;
    the step is captured into a graph and replayed on another stream."""
    torch = torch_mod()
    rng = np.random.default_rng(50)
    H, Hkv, d, prompts, steps = 8, 2, 64, [37, 100, 1], 20
    final = [n + steps for n in prompts]
    c = Cache(final, Hkv, d, seed=51)
    S = len(prompts)
    c.append(fa, *(cr.bf16(rng, sum(prompts), Hkv, d) for _ in "kv"), prompts, prompts)
    c.check("prompts")
    # the prompts' own attention, as chunks over what was written
    q = bf16(cr.bf16(rng, sum(prompts), H, d))
    got = fa.fa_fwd_paged_fp8(q, *c.args(), dev(np.int32(prompts)), dev(cu_of(prompts)),
                              max(prompts), max(prompts))
    check_chunks(*got, q, c, prompts, cu_of(prompts), 0, 0)
    for window, sinks in ((0, 0), (40, 4)):
        q, k, v = (bf16(cr.bf16(rng, S, h, d)) for h in (H, Hkv, Hkv))
        lens, cu = dev(np.int32(prompts)), dev(cu_of([1] * S))
        ws = fa.new_workspace(fa.fa_decode_window_workspace_size(S, H, Hkv, d, max(final), window,
                                                                 sinks))

        def step():
            fa.fa_cache_append_fp8(k, v, *c.args(), lens, cu, 1)
            return fa.fa_decode_paged_fp8(q, *c.args(), lens, max(final), window, sinks,
                                          workspace=ws)
        lens.add_(1)
        ctx = [n + 1 for n in prompts]
        eager = step()  # also the one-time set-up outside the capture
        for x, t in (("k", k), ("v", v)):
            cr.append(t.float().cpu().numpy(), c.pool[x], c.scale[x], c.table, ctx, [1] * S)
        check_decode(*eager, q, c, ctx, window, sinks, "eager")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        side = torch.cuda.Stream()
        for _ in range(steps // 2 - 1):
            ctx = [n + 1 for n in ctx]
            lens.add_(1)
            new = {x: cr.bf16(rng, S, h, d) for x, h in (("q", H), ("k", Hkv), ("v", Hkv))}
            for t, x in ((q, "q"), (k, "k"), (v, "v")):
                t.copy_(bf16(new[x]))
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
            for x in "kv":
                cr.append(new[x], c.pool[x], c.scale[x], c.table, ctx, [1] * S)
            c.check(f"window {window} context {ctx}")
            check_decode(*captured, q, c, ctx, window, sinks, f"context {ctx}")
        prompts = ctx
    assert_device_clean()


def test_two_calls_at_once(fa):
    """Decode calls on two streams with workspaces of their own."""
    torch = torch_mod()
    ctx, H, Hkv, d = [900, 1100], 8, 2, 128
    c = Cache(ctx, Hkv, d, seed=60)
    rng = np.random.default_rng(61)
    qs = [bf16(cr.bf16(rng, 2, H, d)) for _ in range(2)]
    lens = dev(np.int32(ctx))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[] for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            outs[i].append(fa.fa_decode_paged_fp8(qs[i], *c.args(), lens, 1100, stream=s))
    torch.cuda.synchronize()
    assert_device_clean()
    for i in range(2):
        check_decode(*outs[i][0], qs[i], c, ctx, 0, 0, f"stream {i}")
        for o, l in outs[i][1:]:
            assert torch.equal(o, outs[i][0][0]) and torch.equal(l, outs[i][0][1])


def test_binding_refuses(fa):
    torch = torch_mod()
    c = Cache([40], 2, 64, seed=70)
    q = bf16(np.zeros((1, 4, 64), np.float32))
    lens = dev(np.int32([40]))
    for window, sinks in ((-1, 0), (0, 3), (5, -1)):
        with pytest.raises(ValueError):
            fa.fa_decode_paged_fp8(q, *c.args(), lens, 40, window, sinks)
    kp, vp, ks, vs, table = c.args()
    with pytest.raises(ValueError):
        fa.fa_decode_paged_fp8(q, kp, vp, ks[:-1], vs, table, lens, 40)
    with pytest.raises(ValueError):
        fa.fa_decode_paged_fp8(q, kp.float(), vp, ks, vs, table, lens, 40)
    with pytest.raises(ValueError):
        fa.fa_decode_paged_fp8(q, kp, vp, ks.double(), vs, table, lens, 40)
    with pytest.raises(fa.FaError):
        fa.fa_decode_paged_fp8(q, *c.args(), lens, 4000)
    for window, sinks in ((-1, 0), (0, 3)):
        with pytest.raises(ValueError):
            fa.fa_fwd_paged_fp8(q, *c.args(), lens, dev(np.int32([0, 1])), 1, 40, window, sinks)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_fp8(q, *c.args(), lens, dev(np.int32([0])), 1, 40)
    k = bf16(np.zeros((40, 2, 64), np.float32))
    cu = dev(np.int32([0, 40]))
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(k.transpose(1, 2), k, *c.args(), lens, cu, 40)
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(k[:, :, :32], k, *c.args(), lens, cu, 40)
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(k, k[:-1], *c.args(), lens, cu, 40)
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(k[:1].expand(40, 2, 64), k, *c.args(), lens, cu, 40)
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(k, k, *c.args(), lens, cu[:1], 40)


def test_no_rows(fa):
    """A step without tokens does nothing."""
    c = Cache([40], 2, 64, seed=1)
    q, k, lens = bf16(np.zeros((0, 4, 64))), bf16(np.zeros((0, 2, 64))), dev(np.int32([40]))
    cu = dev(np.int32([0, 0]))
    fa.fa_cache_append_fp8(k, k, *c.args(), lens, cu, 0)
    c.check()
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), lens, cu, 0, 40)
    assert out.shape == q.shape and lse.shape == (4, 0)
    out, lse = fa.fa_decode_paged_fp8(q, *c.args()[:4], c.dtable[:0], lens[:0], 40)
    assert out.shape == q.shape and lse.shape == (0, 4)
    assert_device_clean()


def test_blocks_past_32_bits(fa):
    """Blocks whose codes lie past 2^31 and 2^32 bytes of the pool."""
    torch = torch_mod()
    H, Hkv, d, n, new = 16, 8, 128, 155, 30
    c = Cache([n], Hkv, d, seed=130)
    near = c.table.copy()
    base = (1 << 32) // (16 * Hkv * d) - 5   # the ten blocks lie on both sides of 2^32
    size = base + 1 + int(near.max())
    for x in "kv":
        pool = torch.zeros(size, 16, Hkv, d, dtype=torch.uint8, device="cuda")
        pool[base:] = c.dpool[x][:size - base]
        scale = torch.ones(size, Hkv, dtype=torch.float32, device="cuda")
        scale[base:] = c.dscale[x][:size - base]
        c.dpool[x], c.dscale[x] = pool, scale
    c.dtable = dev((near + base).astype(np.int32))
    rng = np.random.default_rng(131)
    k, v = (cr.bf16(rng, new, Hkv, d) for _ in "kv")
    c.append(fa, k, v, [n], [new])
    far = c.dpool, c.dscale
    c.dpool = {x: far[0][x][base:] for x in "kv"}
    c.dscale = {x: far[1][x][base:] for x in "kv"}
    for x in "kv":   # (the twin's blocks behind the table's are not in the pool)
        c.pool[x], c.scale[x] = c.pool[x][:size - base], c.scale[x][:size - base]
    c.check("far blocks")
    assert not any(int(far[0][x][:base].count_nonzero()) for x in "kv")
    c.dpool, c.dscale = far
    q = bf16(cr.bf16(rng, new, H, d))
    lens, cu = dev(np.int32([n])), dev(np.int32([0, new]))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), lens, cu, new, n)
    check_chunks(out, lse, q, c, [n], [0, new], 0, 0)
    out, lse = fa.fa_decode_paged_fp8(q[-1:].contiguous(), *c.args(), lens, n)
    check_decode(out, lse, q[-1:], c, [n], 0, 0, "far blocks")
    assert_device_clean()


@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (6, 3, 128)])
def test_chunks_of_any_size_of_row(fa, H, Hkv, d):
    """Queries of 2^-60 to 2^100 over keys whose block scales make up for it,
    values 2^-8 and 2^-12 of their row's largest, zero rows; rows with an
    infinity or a NaN become NaN and leave the others alone.

    The products hold q to 2^-21 of its row's largest value: a score is off by
    2^-21 max|q| sum|k| of its scale, and the output by twice that (in its
    weights and in their sum) of sum P |v|."""
    torch = torch_mod()
    ctx, new = [300, 170], [150, 40]
    c = Cache(ctx, Hkv, d, seed=140)
    rng = np.random.default_rng(141)
    G = H // Hkv
    size = np.exp2([(-60, 0, 100, 37)[h] for h in range(Hkv)]).astype(np.float32)
    c.scale["k"] = (c.scale["k"] / size).astype(np.float32)
    c.dscale["k"].copy_(dev(c.scale["k"]))
    cu = cu_of(new)
    q = cr.bf16(rng, cu[-1], H, d) * np.repeat(size, G)[:, None]
    q[:, :, 5:] *= np.float32(2.0 ** -8)
    q[:, :, 9:] *= np.float32(2.0 ** -4)
    q[7], q[160] = 0, 0
    q = bf16(q)
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), dev(np.int32(ctx)), dev(cu), max(new), max(ctx))
    assert_device_clean()
    for b, n in enumerate(ctx):
        a, e = int(cu[b]), int(cu[b + 1])
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        for h in range(H):
            x, kh, vh = q[a:e, h].double(), k[:, h // G], v[:, h // G]
            o, l, tol = ref.forward(x, kh, vh, 0, 0)
            off = 2.0 ** -21 * x.abs().amax(1) * kh.abs().sum(1).max() / math.sqrt(d)
            size_v = torch.softmax((x @ kh.T / math.sqrt(d)).masked_fill(
                ~ref.visible(e - a, n, n - (e - a), 0, 0, x.device), -math.inf), 1) @ vh.abs()
            ref.assert_within(out[a:e, h], o, tol + 2 * off[:, None] * size_v, f"seq {b} head {h}")
            assert bool(((lse[h, a:e].double() - l).abs() <= ref.LSE_TOL + off).all()), (b, h)
    bad = q.clone()
    bad[3, 0, 1], bad[151, :, d - 1] = math.inf, math.nan
    got, _ = fa.fa_fwd_paged_fp8(bad, *c.args(), dev(np.int32(ctx)), dev(cu), max(new), max(ctx))
    assert bool(got[3, 0].isnan().all()) and bool(got[151].isnan().all())
    got[3, 0], got[151] = out[3, 0], out[151]
    assert torch.equal(got, out)
    assert_device_clean()


def test_padded_serving_batch(fa):
    """Slots of a batch without a sequence (no tokens, empty context, table row
    of no ids) and rows behind the last sequence: nothing of them is written,
    whatever their rows hold; pools as e4m3 tensors give the same bits."""
    torch = torch_mod()
    H, Hkv, d = 4, 2, 128
    ctx, new = [0, 70, 0, 33, 0], [0, 5, 0, 33, 0]
    c = Cache(ctx, Hkv, d, seed=150)
    rng = np.random.default_rng(151)
    T = sum(new)
    k, v = cr.bf16(rng, T + 4, Hkv, d), cr.bf16(rng, T + 4, Hkv, d)
    k[T:], v[T:] = np.nan, np.nan
    c.append(fa, k, v, ctx, new)
    c.check("padded")
    q = bf16(cr.bf16(rng, T + 4, H, d))
    q[T:] = math.nan
    lens, cu = dev(np.int32(ctx)), dev(cu_of(new))
    for window, sinks in ((0, 0), (20, 3)):
        out = torch.full_like(q, 7.0)
        lse = torch.full((H, T + 4), 7.0, device="cuda")
        fa.fa_fwd_paged_fp8(q, *c.args(), lens, cu, max(new), max(ctx), window, sinks, out=out, lse=lse)
        assert bool((out[T:] == 7.0).all()) and bool((lse[:, T:] == 7.0).all())
        check_chunks(out[:T], lse[:, :T], q[:T], c, ctx, cu_of(new), window, sinks)
        tok = bf16(cr.bf16(rng, len(ctx), H, d))
        got = fa.fa_decode_paged_fp8(tok, *c.args(), lens, max(ctx), window, sinks)
        check_decode(*got, tok, c, ctx, window, sinks, "padded")
        e4m3 = [t.view(torch.float8_e4m3fn) for t in c.args()[:2]]
        same = fa.fa_decode_paged_fp8(tok, *e4m3, *c.args()[2:], lens, max(ctx), window, sinks)
        assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    assert_device_clean()
