"""Calls at the edges of what the windowed and 8-bit cache calls document:
rows that are not finite, very wide block tables, sequences longer than said,
workspaces sized for longer calls, tiny and subnormal queries."""
import math

import numpy as np
import pytest

import cache_reference as cr
import window_reference as ref
from gpu_helpers import assert_device_clean, torch_mod
from test_gpu_kvcache import Cache, bf16, cu_of, dev
from test_gpu_window import check_gradient, check_rows, i32, normal, pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa_mod
    fa_mod.fa_device_status(clear=True)
    return fa_mod


def assert_poisoned(got, want, rows):
    """(out, lse) [rows.., H, d], [rows.., H]: NaN at the (row, head) pairs of
    `rows`, the bits of `want` elsewhere."""
    torch = torch_mod()
    (out, lse), (o, l) = got, want
    for r, h in rows:
        assert bool(out[r, h].isnan().all()), (r, h)
        assert bool(lse[r, h].isnan()), (r, h, float(lse[r, h]))
        out[r, h], lse[r, h] = o[r, h], l[r, h]
    assert torch.equal(out, o) and torch.equal(lse, l)


# ------------------------------------------------------------------ rows that are not finite

@pytest.mark.parametrize("H,Hkv,d,window,sinks", [(4, 2, 64, 0, 0), (32, 2, 128, 0, 0),
                                                  (8, 1, 128, 600, 4), (3, 1, 64, 5, 0)])
def test_tokens_over_codes_with_bad_queries(fa, H, Hkv, d, window, sinks):
    """A query with a NaN or an infinity gets NaN, not what an empty context
    gets; in contexts of one key, one split and many."""
    ctx = [1, 60, 0, 3000]
    c = Cache(ctx, Hkv, d, seed=200)
    q = bf16(cr.bf16(np.random.default_rng(d), len(ctx), H, d))
    args = (*c.args(), dev(np.int32(ctx)), max(ctx), window, sinks)
    want = fa.fa_decode_paged_fp8(q, *args)
    for value in (math.nan, math.inf, -math.inf):
        bad = q.clone()
        rows = [(0, 0), (1, H - 1), (3, 1), (3, 2)]
        for i, (r, h) in enumerate(rows):
            bad[r, h, (7 * i) % d] = value
        assert_poisoned(fa.fa_decode_paged_fp8(bad, *args), want, rows)
    bad = q.clone()
    bad[2] = math.nan     # over no keys: still an empty row
    assert_poisoned(fa.fa_decode_paged_fp8(bad, *args), want, [])
    assert_device_clean()


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (32, 2, 128)])
@pytest.mark.parametrize("window", [0, 50, 2000])
def test_tokens_over_bf16_with_bad_queries(fa, H, Hkv, d, window):
    ctx = [1, 60, 0, 3000]
    kp, vp, table, _ = pages(ctx, Hkv, d, 210)
    q = normal(212, len(ctx), H, d)

    def call(q):
        args = (q, kp, vp, table.cuda(), i32(ctx), max(ctx))
        return fa.fa_decode_paged_window(*args, window, 3) if window else fa.fa_decode_paged(*args)
    want = call(q)
    bad = q.clone()
    bad[0, 0, 1] = bad[1, H - 1, 0] = bad[3, 1, d - 1] = bad[2] = math.nan
    assert_poisoned(call(bad), want, [(0, 0), (1, H - 1), (3, 1)])
    assert_device_clean()


def test_a_bad_key_reaches_its_log_sum_too(fa):
    """A NaN code in a visible key makes the token's output NaN, and its
    log-sum-exp with it."""
    ctx, H, Hkv, d = [100, 100], 4, 2, 64
    c = Cache(ctx, Hkv, d, seed=215)
    q = bf16(cr.bf16(np.random.default_rng(1), 2, H, d))
    args = (*c.args(), dev(np.int32(ctx)), 100)
    want = fa.fa_decode_paged_fp8(q, *args)
    c.dpool["k"][int(c.table[1, 3]), 5, 0, 9] = 0x7F
    assert_poisoned(fa.fa_decode_paged_fp8(q, *args), want, [(1, 0), (1, 1)])
    assert_device_clean()


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (6, 2, 128)])
def test_chunks_and_prompts_with_bad_queries(fa, H, Hkv, d):
    """Rows with a NaN are NaN in out and lse alike, in every windowed and
    8-bit form; so are rows with an infinity over the 8-bit cache."""
    ctx, new = [300, 170], [150, 40]
    cu, T = cu_of(new), sum(new)
    rows = [(3, 0), (151, 1), (151, 2), (189, H - 1)]
    c = Cache(ctx, Hkv, d, seed=220)
    kp, vp, table, _ = pages(ctx, Hkv, d, 221)
    q, k, v = (normal(222 + i, T, h, d) for i, h in enumerate((H, Hkv, Hkv)))
    bad = q.clone()
    for r, h in rows:
        bad[r, h, r % d] = math.nan
    lens, dcu = dev(np.int32(ctx)), dev(cu)
    calls = [
        lambda q: fa.fa_fwd_paged_fp8(q, *c.args(), lens, dcu, max(new), max(ctx)),
        lambda q: fa.fa_fwd_paged_fp8(q, *c.args(), lens, dcu, max(new), max(ctx), 40, 3),
        lambda q: fa.fa_fwd_paged_window(q, kp, vp, table.cuda(), lens, dcu, max(new), max(ctx), 40, 3),
        lambda q: fa.fa_fwd_varlen_window(q, k, v, dcu, max(new), 40, 3),
        lambda q: [t[0] for t in fa.fa_fwd_window(q[None], k[None], v[None], 40, 3)],
    ]
    for i, call in enumerate(calls):
        (out, lse), (o, l) = call(bad), call(q)
        assert_poisoned((out, lse.T.contiguous()), (o, l.T.contiguous()), rows)
        if i < 2:
            inf = q.clone()
            inf[bad.isnan()] = math.inf
            out, lse = call(inf)
            assert_poisoned((out, lse.T.contiguous()), (o, l.T.contiguous()), rows)
    assert_device_clean()


# ------------------------------------------------------------------ sizes

def test_documented_workspace_of_a_gradient(fa):
    """A gradient's workspace sized with the longest sequence, which a batch of
    fewer rows than that does not reach."""
    torch = torch_mod()
    H, Hkv, d, window, sinks, T, said = 4, 4, 128, 1, 300, 256, 257
    cu = i32([0, T])
    q, k, v, g = (normal(250 + i, T, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    out, lse = fa.fa_fwd_varlen_window(q, k, v, cu, said, window, sinks)
    ws = torch.empty(fa.fa_bwd_window_workspace_size(1, H, Hkv, said, d, window, sinks),
                     dtype=torch.uint8, device="cuda")
    grads = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, cu, said, window, sinks, workspace=ws)
    assert_device_clean()
    check_gradient(*grads, q, k, v, g, window, sinks, "shorter than said")


def test_documented_workspace_of_single_tokens(fa):
    """Workspaces sized with the longest context, while contexts are short."""
    H, Hkv, batch = 8, 8, 64
    for window, limit in ((0, 2049), (2040, 8000)):
        sized = fa.fa_decode_window_workspace_size(batch, H, Hkv, 64, limit, window)
        ctx = [40] * batch
        c = Cache(ctx, Hkv, 64, seed=253, width=500)
        q = normal(254, batch, H, 64)
        for longest in (40, 1024, 2048, limit):
            ws = fa.new_workspace(sized)
            got = fa.fa_decode_paged_fp8(q, *c.args(), dev(np.int32(ctx)), longest, window,
                                         workspace=ws)
            for h in range(H):
                o, l, tol = cr.decode_rows(q[:1, h].double(), c.rows("k", 0, 40)[:, h],
                                           c.rows("v", 0, 40)[:, h], window, 0)
                ref.assert_within(got[0][:1, h], o, tol, f"longest {longest}")
    assert_device_clean()


def test_tables_of_many_columns(fa):
    """A table whose columns hold 2^31 tokens and more."""
    torch = torch_mod()
    ctx, H, Hkv, d, width = [90], 4, 2, 64, (1 << 27) + 8
    lens, cu = dev(np.int32(ctx)), dev(np.int32([0, 20]))
    q = normal(231, 20, H, d)
    c = Cache(ctx, Hkv, d, seed=230)
    kp, vp, table, _ = pages(ctx, Hkv, d, 232)
    codes, bf = c.args()[:4], (kp, vp)
    calls = [
        (c.dtable, lambda t: fa.fa_decode_paged_fp8(q[-1:], *codes, t, lens, 90)),
        (c.dtable, lambda t: fa.fa_decode_paged_fp8(q[-1:], *codes, t, lens, 90, 30, 2)),
        (c.dtable, lambda t: fa.fa_fwd_paged_fp8(q, *codes, t, lens, cu, 20, 90)),
        (table.cuda(), lambda t: fa.fa_decode_paged_window(q[-1:], *bf, t, lens, 90, 30, 2)),
        (table.cuda(), lambda t: fa.fa_fwd_paged_window(q, *bf, t, lens, cu, 20, 90, 30, 2)),
        (table.cuda(), lambda t: fa.fa_decode_paged(q[-1:], *bf, t, lens, 90)),
        (table.cuda(), lambda t: fa.fa_fwd_paged(q, *bf, t, lens, cu, 20, 90)),
    ]
    wide = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    for i, (few, call) in enumerate(calls):
        wide[:, :6] = few[:, :6]
        want, got = call(few), call(wide)
        assert_device_clean()
        assert all(torch.equal(x, y) for x, y in zip(want, got)), i
        assert bool(torch.isfinite(got[1]).all()), i


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (3, 3, 128)])
def test_a_sequence_longer_than_said(fa, H, Hkv, d):
    """max_seqlen is a bound on every length; a longer sequence that the launch
    covers all the same keeps its own window."""
    lens, said, window, sinks = [100, 60], 50, 80, 2
    cu = [0, 100, 160]
    q, k, v = (normal(240 + i, 160, h, d) for i, h in enumerate((H, Hkv, Hkv)))
    out, lse = fa.fa_fwd_varlen_window(q, k, v, i32(cu), said, window, sinks)
    assert fa.fa_device_status(clear=True) in (0, fa.FA_DEV_BAD_SEQLEN)
    for a, e in zip(cu, cu[1:]):
        check_rows(out[a:e], lse[:, a:e], q[a:e], k[a:e], v[a:e], window, sinks, f"row {a}")


# ------------------------------------------------------------------ tiny queries

@pytest.mark.parametrize("top", [-100, -119, -122, -126, -128, -133])
def test_tiny_queries_over_large_keys(fa, top):
    """Queries of 2^top, down to bf16's smallest subnormal, over blocks whose
    scales make up for it."""
    ctx, H, Hkv, d, n = [90], 2, 1, 64, 20
    c = Cache(ctx, Hkv, d, seed=260)
    rng = np.random.default_rng(261)
    c.scale["k"] = np.full_like(c.scale["k"], 2.0 ** min(-top - 8, 118))
    c.dscale["k"].copy_(dev(c.scale["k"]))
    # few significand bits: also the subnormal ones are exact
    x = rng.integers(-3, 4, (n, H, d)).astype(np.float64) * 2.0 ** top
    q = bf16(x.astype(np.float32))
    assert np.array_equal(q.float().cpu().numpy().astype(np.float64), x)
    lens, cu = dev(np.int32(ctx)), dev(np.int32([0, n]))
    out, lse = fa.fa_fwd_paged_fp8(q, *c.args(), lens, cu, n, 90)
    tok, tlse = fa.fa_decode_paged_fp8(q[-1:], *c.args(), lens, 90)
    assert_device_clean()
    k, v = c.rows("k", 0, 90)[:, 0], c.rows("v", 0, 90)[:, 0]
    for h in range(H):
        qh = dev(x[:, h])
        o, l, tol = ref.forward(qh, k, v, 0, 0)
        # scores: fp32 sums of exact products
        off = 2.0 ** -18 * float((qh.abs() @ k.T.abs()).max()) / math.sqrt(d)
        size = 2 * off * float(v.abs().max())
        ref.assert_within(out[:, h], o, tol + size, f"chunk head {h}")
        assert float((lse[h].double() - l).abs().max()) <= ref.LSE_TOL + off
        o, l, tol = cr.decode_rows(qh[-1:], k, v, 0, 0)
        ref.assert_within(tok[:, h], o, tol + size, f"token head {h}")
        assert abs(float(tlse[0, h]) - float(l)) <= ref.LSE_TOL + off


# ------------------------------------------------------------------ what a call takes

def allocations(call):
    torch = torch_mod()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats().get("allocation.all.allocated", 0)
    keep = call()
    return torch.cuda.memory_stats()["allocation.all.allocated"] - before, keep


def test_calls_allocate_their_outputs_once(fa):
    ctx, H, Hkv, d = [90, 40], 4, 2, 64
    c = Cache(ctx, Hkv, d, seed=270)
    kp, vp, table, _ = pages(ctx, Hkv, d, 271)
    table, lens = table.cuda(), i32(ctx)
    tok = normal(272, 2, H, d)
    q, k, v, g = (normal(273 + i, 1, 90, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    cu = i32([0, 90])
    out, lse = fa.fa_fwd_window(q, k, v, 30, 2)
    calls = [   # outputs and the workspace
        (3, lambda: fa.fa_decode_paged_fp8(tok, *c.args(), lens, 90)),
        (3, lambda: fa.fa_decode_paged_window(tok, kp, vp, table, lens, 90, 30, 2)),
        (4, lambda: fa.fa_bwd_window(q, k, v, out, lse, g, 30, 2)),
        (4, lambda: fa.fa_bwd_varlen_window(q[0], k[0], v[0], out[0], lse[0], g[0], cu, 90, 30, 2)),
    ]
    for i, (most, call) in enumerate(calls):
        call()
        n, _ = allocations(call)
        assert n <= most, (i, n)
    assert_device_clean()


def test_gradient_without_the_output(fa):
    """The windowed gradient forms its row sums itself: O may be gone."""
    torch = torch_mod()
    lens, H, Hkv, d, window, sinks = [90, 200], 4, 2, 64, 30, 2
    cu = i32([0, 90, 290])
    q, k, v, g = (normal(280 + i, 290, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    out, lse = fa.fa_fwd_varlen_window(q, k, v, cu, 200, window, sinks)
    want = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, cu, 200, window, sinks)
    got = fa.fa_bwd_varlen_window(q, k, v, None, lse, g, cu, 200, window, sinks)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ws = torch.empty(fa.fa_bwd_window_workspace_size(2, H, Hkv, 200, d, window, sinks),
                     dtype=torch.uint8, device="cuda")
    got = fa.fa_bwd_varlen_window(q, k, v, None, lse, g, cu, 200, window, sinks, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    q, k, v, g = (t[None, :200].contiguous() for t in (q, k, v, g))
    out, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    want = fa.fa_bwd_window(q, k, v, out, lse, g, window, sinks)
    got = fa.fa_bwd_window(q, k, v, None, lse, g, window, sinks)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(ValueError):
        fa.fa_bwd_window(q, k, v, out[:, :50], lse, g, window, sinks)
    assert_device_clean()
