"""Windowed attention with sinks (fa_*_window) against 64-bit arithmetic:
every layout, the lengths, windows and sinks at which tiles, blocks and masks
meet, rows that see nothing, freed cache blocks, hidden values that are NaN,
other streams and graphs."""
import math

import pytest

import window_reference as ref
from gpu_helpers import assert_device_clean, torch_mod

pytestmark = pytest.mark.gpu

BF16 = dict(device="cuda")


@pytest.fixture(scope="module")
def fa():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa_mod
    fa_mod.fa_device_status(clear=True)
    return fa_mod


def normal(seed, *shape):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def i32(values):
    torch = torch_mod()
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def check_rows(out, lse, q, k, v, window, sinks, what):
    """out [n, H, d], lse [H, n] of queries that are the last n of k's rows."""
    H, Hkv = q.shape[1], k.shape[1]
    for h in range(H):
        kv = h // (H // Hkv)
        o, l, tol = ref.forward(q[:, h].double(), k[:, kv].double(), v[:, kv].double(), window, sinks)
        ref.assert_within(out[:, h], o, tol, f"{what} head {h}")
        ref.assert_lse(lse[h], l, f"{what} head {h}")


# (B, N, H, Hkv, d, window, sinks)
DENSE = [
    (1, 1, 1, 1, 64, 1, 0),
    (2, 1, 4, 2, 128, 7, 3),
    (1, 2, 3, 3, 128, 1, 0),
    (2, 300, 4, 2, 128, 64, 4),      # head pairs
    (1, 517, 6, 3, 64, 100, 0),
    (1, 700, 3, 1, 64, 130, 130),    # group of 3: one tile per CTA
    (1, 640, 2, 2, 128, 128, 0),     # tile-sized windows
    (1, 640, 2, 1, 128, 129, 1),
    (1, 640, 2, 2, 64, 127, 127),
    (1, 1025, 8, 1, 128, 257, 200),  # sinks beyond one tile
    (1, 900, 2, 2, 64, 1, 0),        # each query its own key
    (1, 900, 2, 1, 128, 1, 5),
    (1, 800, 7, 7, 128, 5000, 3),    # longer than the sequence: plain causal
    (1, 450, 2, 1, 64, 20, 9000),    # sinks cover everything
    (1, 1300, 4, 1, 128, 300, 0),
]


@pytest.mark.parametrize("B,N,H,Hkv,d,window,sinks", DENSE)
def test_dense(fa, B, N, H, Hkv, d, window, sinks):
    q, k, v = normal(1, B, N, H, d), normal(2, B, N, Hkv, d), normal(3, B, N, Hkv, d)
    out, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    assert_device_clean()
    for b in range(B):
        check_rows(out[b], lse[b], q[b], k[b], v[b], window, sinks, f"batch {b}")


@pytest.mark.parametrize("B,N,H,Hkv,d,window,sinks", DENSE)
def test_dense_gradient(fa, B, N, H, Hkv, d, window, sinks):
    torch = torch_mod()
    q, k, v = normal(4, B, N, H, d), normal(5, B, N, Hkv, d), normal(6, B, N, Hkv, d)
    g = normal(7, B, N, H, d)
    out, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    dq, dk, dv = fa.fa_bwd_window(q, k, v, out, lse, g, window, sinks)
    assert_device_clean()
    for b in range(B):
        check_gradient(dq[b], dk[b], dv[b], q[b], k[b], v[b], g[b], window, sinks, f"batch {b}")
    if window == 1 and sinks == 0:  # a softmax of one key does not move
        assert not dq.any() and not dk.any()


def check_gradient(dq, dk, dv, q, k, v, g, window, sinks, what):
    torch = torch_mod()
    H, Hkv = q.shape[1], k.shape[1]
    G = H // Hkv
    for kv in range(Hkv):
        sums = [torch.zeros_like(k[:, kv], dtype=torch.float64) for _ in range(4)]
        for h in range(kv * G, kv * G + G):
            (rq, rk, rv), (tq, tk, tv) = ref.backward(q[:, h].double(), k[:, kv].double(),
                                                      v[:, kv].double(), g[:, h].double(), window,
                                                      sinks)
            ref.assert_within(dq[:, h], rq, tq, f"{what} dq {h}")
            # each head's tolerance counts the rounding of its own share; the
            # sum is rounded once, by no more than those together
            for s, x in zip(sums, (rk, tk, rv, tv)):
                s += x
        sums[1] += ref.U * sums[0].abs()
        sums[3] += ref.U * sums[2].abs()
        ref.assert_within(dk[:, kv], sums[0], sums[1], f"{what} dk {kv}")
        ref.assert_within(dv[:, kv], sums[2], sums[3], f"{what} dv {kv}")


PACKED = [
    ([5, 1, 0, 129, 300, 128, 2], 4, 2, 128, 50, 4),
    ([1, 1, 1], 2, 2, 64, 3, 1),
    ([700, 64, 511], 3, 1, 64, 200, 17),
    ([257, 900], 8, 8, 128, 128, 0),
    ([40] * 150, 2, 1, 64, 16, 2),            # beyond the padding-free order
    ([33, 1500, 7], 4, 1, 128, 1000, 300),
]


@pytest.mark.parametrize("lens,H,Hkv,d,window,sinks", PACKED)
def test_packed_with_gradient(fa, lens, H, Hkv, d, window, sinks):
    """Rows behind the last sequence hold NaN and keep what the outputs held."""
    torch = torch_mod()
    cu = cu_of(lens)
    t, extra = cu[-1], 37
    q, k, v, g = (normal(8 + i, t + extra, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    for x in (q, k, v, g):
        x[t:] = math.nan
    out, lse = torch.full_like(q, 3.0), torch.full((H, t + extra), 3.0, device="cuda")
    fa.fa_fwd_varlen_window(q, k, v, i32(cu), max(lens), window, sinks, out=out, lse=lse)
    dq, dk, dv = (torch.full_like(x, 3.0) for x in (q, k, v))
    fa.fa_bwd_varlen_window(q, k, v, out, lse, g, i32(cu), max(lens), window, sinks, dq=dq, dk=dk,
                            dv=dv)
    assert_device_clean()
    for x in (out, dq, dk, dv):
        assert (x[t:] == 3).all()
    assert (lse[:, t:] == 3).all()
    for a, b in list(zip(cu, cu[1:]))[:8]:
        if a == b:
            continue
        r = slice(a, b)
        check_rows(out[r], lse[:, r], q[r], k[r], v[r], window, sinks, f"rows {a}:{b}")
        check_gradient(dq[r], dk[r], dv[r], q[r], k[r], v[r], g[r], window, sinks, f"rows {a}:{b}")


# more work items than SMs, behind one another in the same CTAs
MANY = [
    ([2048, 2048], 16, 4, 128, 200, 5),
    ([4096], 32, 8, 64, 129, 0),
    ([1500, 3, 0, 700, 2900, 1, 129, 128], 16, 4, 128, 300, 140),
    ([3000] + [40] * 140, 8, 2, 64, 100, 3),        # beyond the padding-free order
    ([1300, 1, 1291], 24, 4, 128, 1, 0),
]


@pytest.mark.parametrize("lens,H,Hkv,d,window,sinks", MANY)
def test_many_items(fa, lens, H, Hkv, d, window, sinks):
    torch = torch_mod()
    cu = cu_of(lens)
    q, k, v = (normal(140 + i, cu[-1] + 3, h, d) for i, h in enumerate((H, Hkv, Hkv)))
    q[-3:], k[-3:], v[-3:] = math.nan, math.nan, math.nan     # of no sequence
    out = torch.full_like(q, 7.0)
    _, lse = fa.fa_fwd_varlen_window(q, k, v, i32(cu), max(lens), window, sinks, out=out)
    assert_device_clean()
    assert bool((out[-3:] == 7.0).all())
    for n in sorted(set(lens)):
        a = cu[lens.index(n)]
        if n:
            check_rows(out[a:a + n], lse[:, a:a + n], q[a:a + n], k[a:a + n], v[a:a + n], window,
                       sinks, f"{n} rows")
    if lens[0] == lens[-1]:
        q, k, v = (t[:-3].reshape(len(lens), lens[0], -1, d) for t in (q, k, v))
        dense, dlse = fa.fa_fwd_window(q, k, v, window, sinks)
        assert_device_clean()
        for b in range(len(lens)):
            check_rows(dense[b], dlse[b], q[b], k[b], v[b], window, sinks, f"dense {b}")


def test_bad_sequence_among_many(fa):
    """A sequence with bad bounds is reported and passed over; the CTAs that meet
    it go on."""
    torch = torch_mod()
    for count in (3, 140):                       # with and beyond the padding-free order
        lens = [1500] + [30] * (count - 3) + [1500, 300]
        cu = cu_of(lens)
        q, k, v = (normal(150 + i, cu[-1], h, 128) for i, h in enumerate((16, 4, 4)))
        bad = list(cu)
        bad[-1] += 1                             # the last ends past the rows
        out, lse = fa.fa_fwd_varlen_window(q, k, v, i32(bad), 1500, 200, 4)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_SEQLEN
        for a, e in ((cu[0], cu[1]), (cu[-3], cu[-2])):
            check_rows(out[a:e], lse[:, a:e], q[a:e], k[a:e], v[a:e], 200, 4, f"{count}, row {a}")


def test_values_of_another_sequence_do_not_matter(fa):
    """A sequence next to one of infinities and NaN gives the same bits."""
    torch = torch_mod()
    lens, H, Hkv, d = [100, 300, 77], 4, 2, 64
    cu, t = i32(cu_of(lens)), sum(lens)
    q, k, v, g = (normal(20 + i, t, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))

    def run():
        out, lse = fa.fa_fwd_varlen_window(q, k, v, cu, 300, 60, 4)
        return [out, *fa.fa_bwd_varlen_window(q, k, v, out, lse, g, cu, 300, 60, 4)]
    before = [x.clone() for x in run()]
    for x in (q, k, v, g):
        x[100:400:3] = math.nan
        x[101:400:3] = math.inf
    after = run()
    for x, y in zip(before, after):
        assert torch.equal(x[:100], y[:100]) and torch.equal(x[400:], y[400:])


def test_gradient_follows_differences(fa):
    """sum(grad * u) against a central difference of the 64-bit loss."""
    torch = torch_mod()
    N, H, Hkv, d, window, sinks = 260, 4, 2, 64, 70, 6
    q, k, v, g = (normal(30 + i, 1, N, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    out, lse = fa.fa_fwd_window(q, k, v, window, sinks)
    grads = fa.fa_bwd_window(q, k, v, out, lse, g, window, sinks)

    def loss(q, k, v):
        return sum(float((ref.forward(q[0, :, h], k[0, :, h // 2], v[0, :, h // 2], window,
                                      sinks)[0] * g[0, :, h].double()).sum()) for h in range(H))
    x = [t.double() for t in (q, k, v)]
    for i in range(3):
        u = normal(40 + i, *x[i].shape).double()
        step = [t + 1e-4 * u if j == i else t for j, t in enumerate(x)]
        back = [t - 1e-4 * u if j == i else t for j, t in enumerate(x)]
        want = (loss(*step) - loss(*back)) / 2e-4
        got = float((grads[i].double() * u).sum())
        # the gradient's tolerance, against |u|, plus the difference's own h^2
        tol = 0.0
        for h in range(H):
            t = ref.backward(*(y[0, :, h // 2 if j in (1, 2) else h] for j, y in
                               enumerate((*x, g.double()))), window, sinks)[1][i]
            tol += float((t * u[0, :, h if i == 0 else h // 2].abs()).sum())
        assert abs(got - want) <= tol + 1e-4 * abs(want), (i, got, want, tol)


# ------------------------------------------------------------------ cached forms

def pages(ctx, Hkv, d, seed, freed=0, poison=False):
    """A pool of 16-token blocks, its table (unused entries -1), and each
    sequence's keys and values in a row."""
    torch = torch_mod()
    blocks = [(c + 15) // 16 for c in ctx]
    total = sum(blocks) + 2
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(ctx), max(max(blocks), 1)), -1, dtype=torch.int32)
    kp, vp = normal(seed, total, 16, Hkv, d), normal(seed + 1, total, 16, Hkv, d)
    rows = []
    for b, n in enumerate(blocks):
        mine = [perm.pop() for _ in range(n)]
        table[b, :n] = torch.tensor(mine, dtype=torch.int32)
        at = torch.tensor(mine, device="cuda", dtype=torch.long)
        rows.append((kp[at].flatten(0, 1)[:ctx[b]].clone(), vp[at].flatten(0, 1)[:ctx[b]].clone()))
        if ctx[b] % 16:
            kp[mine[-1], ctx[b] % 16:] = math.nan  # stale slots
            vp[mine[-1], ctx[b] % 16:] = math.nan
    return kp, vp, table, rows


DECODE = [
    ([1], 1, 1, 64, 1, 0),
    ([5, 16, 17, 0, 300], 4, 2, 128, 16, 4),
    ([700, 33, 1024], 8, 1, 64, 100, 20),
    ([1000, 999, 15], 6, 2, 128, 1, 0),
    ([2000, 1], 32, 2, 128, 513, 1),          # group of 16
    ([640, 641, 655, 656], 2, 2, 64, 64, 16),
    ([300, 40], 3, 1, 64, 10000, 2),
    ([900], 4, 4, 128, 30, 5000),
    ([5000, 130], 8, 2, 128, 4096, 64),
]


@pytest.mark.parametrize("ctx,H,Hkv,d,window,sinks", DECODE)
def test_decode(fa, ctx, H, Hkv, d, window, sinks):
    """Blocks without a visible key are freed (no table entry) and hidden
    slots of the others hold NaN."""
    kp, vp, table, rows = pages(ctx, Hkv, d, 50)
    for b, c in enumerate(ctx):
        for blk in range((c + 15) // 16):
            tok = [t for t in range(blk * 16, min(c, blk * 16 + 16))]
            hidden = [t for t in tok if t < c - window and t >= sinks]
            phys = int(table[b, blk])
            if len(hidden) == len(tok):
                table[b, blk] = 1 << 30
            for t in hidden:
                kp[phys, t % 16] = vp[phys, t % 16] = math.nan
    q = normal(52, len(ctx), H, d)
    out, lse = fa.fa_decode_paged_window(q, kp, vp, table.cuda(), i32(ctx), max(ctx), window, sinks)
    assert_device_clean()
    for b, c in enumerate(ctx):
        check_rows(out[b:b + 1], lse[b][:, None], q[b:b + 1], *rows[b], window, sinks, f"seq {b}")


CHUNKS = [
    ([5], [5], 2, 1, 64, 3, 1),
    ([300, 129, 40], [100, 129, 1], 4, 2, 128, 64, 4),
    ([700, 16], [20, 3], 3, 3, 64, 200, 20),
    ([1000, 30], [300, 40], 8, 2, 128, 128, 0),   # a chunk longer than its context
    ([2000, 0], [256, 2], 4, 1, 128, 500, 140),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,d,window,sinks", CHUNKS)
def test_paged_chunks(fa, ctx, new, H, Hkv, d, window, sinks):
    kp, vp, table, rows = pages(ctx, Hkv, d, 60)
    for b, (c, n) in enumerate(zip(ctx, new)):
        for blk in range((c + 15) // 16):  # freed: behind the first query's window
            if blk * 16 >= sinks and blk * 16 + 16 <= c - n + 1 - window:
                table[b, blk] = -7
    cu = cu_of(new)
    q = normal(62, cu[-1], H, d)
    out, lse = fa.fa_fwd_paged_window(q, kp, vp, table.cuda(), i32(ctx), i32(cu), max(new), max(ctx),
                                      window, sinks)
    assert_device_clean()
    for b, (a, e) in enumerate(zip(cu, cu[1:])):
        check_rows(out[a:e], lse[:, a:e], q[a:e], *rows[b], window, sinks, f"seq {b}")


def test_prompt_then_tokens(fa):
    """A prompt by the packed call, its chunks over the cache and the tokens
    after it by the decode call agree on what they share."""
    torch = torch_mod()
    n, H, Hkv, d, window, sinks = 333, 4, 2, 128, 90, 5
    kp, vp, table, rows = pages([n], Hkv, d, 70)
    q = normal(72, n, H, d)
    k, v = rows[0]
    out, lse = fa.fa_fwd_varlen_window(q, k, v, i32([0, n]), n, window, sinks)
    part, plse = fa.fa_fwd_paged_window(q[200:], kp, vp, table.cuda(), i32([n]), i32([0, n - 200]),
                                        n - 200, n, window, sinks)
    last, llse = fa.fa_decode_paged_window(q[-1:], kp, vp, table.cuda(), i32([n]), n, window, sinks)
    check_rows(out, lse, q, k, v, window, sinks, "prompt")
    check_rows(part, plse, q[200:], k, v, window, sinks, "chunk")
    check_rows(last, llse.T, q[-1:], k, v, window, sinks, "token")


def test_bad_cache_entries_are_reported(fa):
    """Ids outside the pool and context lengths beyond the table set their
    status bits; the sequences beside them are right."""
    torch = torch_mod()
    ctx, H, Hkv, d = [100, 200, 64], 4, 2, 64
    kp, vp, table, rows = pages(ctx, Hkv, d, 80)
    table[0, 6] = 10 ** 6  # inside the window
    lens = i32([100, 200, 1 << 20])
    q = normal(82, 3, H, d)
    ws = fa.new_workspace(fa.fa_decode_window_workspace_size(3, H, Hkv, d, 200, 40, 4))
    out, lse = fa.fa_decode_paged_window(q, kp, vp, table.cuda(), lens, 200, 40, 4, workspace=ws)
    torch.cuda.synchronize()
    bits = fa.FA_DEV_BAD_BLOCK | fa.FA_DEV_BAD_CTX
    assert fa.fa_last_device_status(ws) == bits
    assert fa.fa_device_status(clear=True) == bits
    check_rows(out[1:2], lse[1][:, None], q[1:2], *rows[1], 40, 4, "seq 1")


# ------------------------------------------------------------------ streams and graphs

def test_other_stream_and_graph(fa):
    """A training step and a decode step on another stream, then captured and
    replayed on new inputs; two graphs with workspaces of their own."""
    torch = torch_mod()
    N, H, Hkv, d, window, sinks = 300, 4, 2, 64, 100, 4
    q, k, v, g = (normal(90 + i, 1, N, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = fa.fa_fwd_window(q, k, v, window, sinks, stream=side)
    grads = fa.fa_bwd_window(q, k, v, out, lse, g, window, sinks, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_rows(out[0], lse[0], q[0], k[0], v[0], window, sinks, "side stream")
    check_gradient(*(x[0] for x in (*grads, q, k, v, g)), window, sinks, "side stream")

    ctx = [N, 37]
    kp, vp, table, rows = pages(ctx, Hkv, d, 96)
    table, lens, tok = table.cuda(), i32(ctx), normal(98, 2, H, d)
    ws = [fa.new_workspace(fa.fa_decode_window_workspace_size(2, H, Hkv, d, N, window, sinks))
          for _ in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, l = fa.fa_fwd_window(q, k, v, window, sinks)
            gr = fa.fa_bwd_window(q, k, v, o, l, g, window, sinks)
            t = fa.fa_decode_paged_window(tok, kp, vp, table, lens, N, window, sinks,
                                          workspace=ws[i])
        graphs.append(graph)
        outs.append((o, l, gr, t))
    for x, s in ((q, 101), (k, 102), (v, 103), (g, 104)):
        x.copy_(normal(s, *x.shape))
    tok.copy_(normal(105, *tok.shape))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert_device_clean()
    for o, l, gr, t in outs:
        check_rows(o[0], l[0], q[0], k[0], v[0], window, sinks, "graph")
        check_gradient(*(x[0] for x in (*gr, q, k, v, g)), window, sinks, "graph")
        for b in range(2):
            check_rows(t[0][b:b + 1], t[1][b][:, None], tok[b:b + 1], *rows[b], window, sinks, "graph")


def test_repeated_calls_give_the_same_bits(fa):
    torch = torch_mod()
    q, k, v, g = (normal(110 + i, 2, 700, h, 128) for i, h in enumerate((8, 2, 2, 8)))
    runs = []
    for _ in range(3):
        out, lse = fa.fa_fwd_window(q, k, v, 150, 130)
        runs.append([out, lse, *fa.fa_bwd_window(q, k, v, out, lse, g, 150, 130)])
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))


def test_binding_refuses(fa):
    torch = torch_mod()
    q, k = normal(1, 1, 8, 4, 64), normal(2, 1, 8, 2, 64)
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(ValueError):
            fa.fa_fwd_window(q, k, k, window, sinks)
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q, k[:, :7], k, 4)
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q.transpose(1, 2), k, k, 4)
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q.float(), k, k, 4)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_window(q[..., :32].contiguous(), k[..., :32].contiguous(),
                         k[..., :32].contiguous(), 4)
    out, lse = fa.fa_fwd_window(q, k, k, 4)
    with pytest.raises(fa.FaError):
        fa.fa_bwd_window(q, k, k, out, lse, out, 4,
                         workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.fa_bwd_window(q, k, k, out, lse[:, :, :4], out, 4)


def test_no_rows(fa):
    """Empty batches and prompts are calls that do nothing."""
    torch = torch_mod()
    for shape in ((0, 5), (3, 0)):
        q, k = normal(1, *shape, 4, 64), normal(2, *shape, 2, 64)
        out, lse = fa.fa_fwd_window(q, k, k, 4)
        assert out.shape == q.shape and lse.shape == (shape[0], 4, shape[1])
        dq, dk, dv = fa.fa_bwd_window(q, k, k, out, lse, q, 4)
        assert dq.shape == q.shape and dk.shape == k.shape and dv.shape == k.shape
    q, k, cu = normal(1, 0, 4, 64), normal(2, 0, 2, 64), i32([0, 0])
    out, lse = fa.fa_fwd_varlen_window(q, k, k, cu, 0, 4, 1)
    assert out.shape == q.shape and lse.shape == (4, 0)
    assert fa.fa_bwd_varlen_window(q, k, k, out, lse, q, cu, 0, 4, 1)[1].shape == k.shape
    pool, table = normal(3, 4, 16, 2, 64), i32([[0, 1]])
    out, lse = fa.fa_fwd_paged_window(q, pool, pool, table, i32([20]), cu, 0, 20, 4)
    assert out.shape == q.shape and lse.shape == (4, 0)
    out, lse = fa.fa_decode_paged_window(q, pool, pool, table[:0], i32([]), 20, 4)
    assert out.shape == q.shape and lse.shape == (0, 4)
    assert_device_clean()


def test_rows_past_32_bits(fa):
    """Rows of q, out and their gradients whose offsets pass 2^31 elements, and
    cache blocks whose offsets do."""
    torch = torch_mod()
    H, Hkv, d, window, sinks = 128, 1, 128, 70, 3
    lens = [(1 << 31) // (H * d) + 5, 260]   # the second sequence lies past 2^31
    cu = cu_of(lens)
    q = normal(120, 4096, H, d).repeat(cu[-1] // 4096 + 1, 1, 1)[:cu[-1]]
    k, v = normal(121, cu[-1], Hkv, d), normal(122, cu[-1], Hkv, d)
    args = (i32(cu), max(lens), window, sinks)
    out, lse = fa.fa_fwd_varlen_window(q, k, v, *args)
    a = cu[1]
    check_rows(out[a:, ::32], lse[::32, a:], q[a:, ::32], k[a:], v[a:], window, sinks, "far rows")
    g = q.flip(0)
    dq, dk, dv = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, *args)
    check_gradient(dq[a:], dk[a:], dv[a:], q[a:], k[a:], v[a:], g[a:], window, sinks, "far rows")
    del q, out, g, dq
    blocks = (1 << 31) // (16 * 8 * d) + 40
    pool = torch.zeros(blocks, 16, 8, d, dtype=torch.bfloat16, device="cuda")
    pool[-20:] = normal(123, 20, 16, 8, d)
    table, n = i32([list(range(blocks - 10, blocks))]), 155
    rows = pool[-10:].reshape(-1, 8, d)[:n]
    tok = normal(124, 30, 16, d)
    o, l = fa.fa_decode_paged_window(tok[-1:], pool, pool, table, i32([n]), n, 100, 2)
    check_rows(o, l[0][:, None], tok[-1:], rows, rows, 100, 2, "far blocks, token")
    o, l = fa.fa_fwd_paged_window(tok, pool, pool, table, i32([n]), i32([0, 30]), 30, n, 100, 2)
    check_rows(o, l, tok, rows, rows, 100, 2, "far blocks, chunk")
    assert_device_clean()


def test_gradient_under_load(fa):
    """Many short work items behind one another, again and again: no wait of the
    pipeline may miss its turn (a missed one raises the status word after a
    second)."""
    torch = torch_mod()
    H, d, lens = 64, 128, [40000, 260]
    q, g = normal(130, sum(lens), H, d), normal(131, sum(lens), H, d)
    k, v = normal(132, sum(lens), 1, d), normal(133, sum(lens), 1, d)
    args = (i32(cu_of(lens)), max(lens), 70, 3)
    out, lse = fa.fa_fwd_varlen_window(q, k, v, *args)
    first = None
    for _ in range(12):
        grads = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, *args)
        first = first or grads
        assert_device_clean()
    assert all(torch.equal(a, b) for a, b in zip(grads, first))


def test_sinks_of_one_long_sequence_among_many(fa):
    """Few slices of the sinks' queries for each sequence: longer ones."""
    H, Hkv, d, window, sinks, n = 2, 2, 64, 16, 2, 4000
    lens = [n] + [1] * 599
    cu = cu_of(lens)
    q, k, v, g = (normal(160 + i, cu[-1], h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    args = (i32(cu), n, window, sinks)
    out, lse = fa.fa_fwd_varlen_window(q, k, v, *args)
    dq, dk, dv = fa.fa_bwd_varlen_window(q, k, v, out, lse, g, *args)
    assert_device_clean()
    for a, e in ((0, n), (n, n + 1), (cu[-2], cu[-1])):
        check_gradient(*(t[a:e] for t in (dq, dk, dv, q, k, v, g)), window, sinks, f"row {a}")


def test_padded_chunks_and_gradients(fa):
    """Rows behind the last sequence, of chunks and of gradients, stay as they
    were, and what they hold reaches nothing."""
    torch = torch_mod()
    H, Hkv, d, window, sinks, pad = 4, 2, 64, 30, 3, 5
    ctx, new = [0, 150, 40], [0, 60, 1]
    kp, vp, table, rows = pages(ctx, Hkv, d, 170)
    q = normal(171, sum(new) + pad, H, d)
    q[-pad:] = math.nan
    out = torch.full_like(q, 7.0)
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    fa.fa_fwd_paged_window(q, kp, vp, table.cuda(), i32(ctx), i32(cu_of(new)), max(new), max(ctx),
                           window, sinks, out=out, lse=lse)
    assert bool((out[-pad:] == 7.0).all()) and bool((lse[:, -pad:] == 7.0).all())
    a = 0
    for n, kv in zip(new, rows):
        if n:
            check_rows(out[a:a + n], lse[:, a:a + n], q[a:a + n], *kv, window, sinks, f"chunk of {n}")
        a += n
    lens = [200, 0, 131]
    cu, T = cu_of(lens), sum(lens)
    q, k, v, g = (normal(172 + i, T + pad, h, d) for i, h in enumerate((H, Hkv, Hkv, H)))
    for t in (q, k, v, g):
        t[-pad:] = math.nan
    out = torch.full_like(q, math.nan)
    _, lse = fa.fa_fwd_varlen_window(q, k, v, i32(cu), 200, window, sinks, out=out)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    fa.fa_bwd_varlen_window(q, k, v, out, lse, g, i32(cu), 200, window, sinks,
                            dq=grads[0], dk=grads[1], dv=grads[2])
    assert_device_clean()
    assert all(bool((t[-pad:] == 7.0).all()) for t in grads)
    for a, e in zip(cu, cu[1:]):
        if e > a:
            check_gradient(*(t[a:e] for t in (*grads, q, k, v, g)), window, sinks, f"rows {a}")
