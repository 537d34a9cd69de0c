"""Single tokens over shared prefixes on the GPU, against attention over each
sequence's own keys in 64 bits."""
import math

import numpy as np
import pytest

import cache_reference as cr
import rope_reference as rr
import window_reference as ref
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


class Batch:
    """Groups as (prefix, [context lengths]); a context may be shorter than the
    prefix.  Sequences of a group share the blocks of its whole ones.  With
    `shared` the table and max_prefix_len are wide enough that the call does not
    take every key as a sequence's own, which it does for few of them."""

    def __init__(self, groups, H, Hkv, d, seed, spread=1.0, shared=True):
        torch = torch_mod()
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.groups, self.H, self.Hkv, self.d = groups, H, Hkv, d
        self.ctx = [c for _, cs in groups for c in cs]
        rows, total = [], 0
        for p, cs in groups:
            common = list(range(total, total + p // 16))
            total += len(common)
            for c in cs:
                mine = max(0, (c + 15) // 16 - len(common))
                rows.append(common + list(range(total, total + mine)))
                total += mine
        perm = rng.permutation(total + 3)
        self.table = np.full((len(rows), max(1, *map(len, rows))), -1, dtype=np.int32)
        for b, r in enumerate(rows):
            self.table[b, :len(r)] = perm[r]
        normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.kp, self.vp = (normal(total + 3, 16, Hkv, d) for _ in "kv")
        self.kp.view(-1, Hkv, d)[::37] *= 4   # maxima that move late
        self.q = normal(len(rows), H, d) * spread
        self.cu = np.concatenate([[0], np.cumsum([len(cs) for _, cs in groups])]).astype(np.int32)
        self.pre = np.int32([p for p, _ in groups])
        self.max_pre = int(max(self.pre, default=0))
        self.max_own = max([max(0, c - p) for p, cs in groups for c in cs], default=0)
        if shared:
            self.max_pre = max(self.max_pre, (64 << 20) // (4 * Hkv * d * len(rows)) + 16)
            more = (self.max_pre + 15) // 16 - self.table.shape[1]
            self.table = np.pad(self.table, ((0, 0), (0, max(0, more))), constant_values=-1)

    def args(self, **new):
        a = dict(q=self.q, k_pool=self.kp, v_pool=self.vp, block_table=dev(self.table),
                 ctx_lens=dev(np.int32(self.ctx)), cu_groups=dev(self.cu), prefix_lens=dev(self.pre),
                 max_prefix_len=self.max_pre, max_own_len=self.max_own)
        return {**a, **new}

    def rows(self, pool, b):
        c = self.ctx[b]
        return pool[dev(self.table[b, : (c + 15) // 16].astype(np.int64))].double().flatten(0, 1)[:c]

    def check(self, out, lse, only=None, scale=None, what=""):
        G = self.H // self.Hkv
        for b in range(len(self.ctx)) if only is None else only:
            k, v = self.rows(self.kp, b), self.rows(self.vp, b)
            for h in range(self.Hkv):
                heads = slice(h * G, h * G + G)
                want, wl, tol = ref.forward(self.q[b, heads].double(), k[:, h], v[:, h], 0, 0,
                                            first=self.ctx[b], scale=scale)
                ref.assert_within(out[b, heads], want, tol, f"{what} sequence {b} head {h}")
                if lse is not None:
                    ref.assert_lse(lse[b, heads], wl, f"{what} sequence {b} head {h}")


CASES = [  # groups (prefix, contexts), H, Hkv, d
    ([(16, [17])], 1, 1, 64),
    ([(0, [5, 40])], 4, 2, 64),                       # nothing shared
    ([(15, [16, 31, 200])], 8, 2, 128),               # less than a block
    ([(1001, [1002, 1040, 1001])], 8, 2, 64),         # a prefix that ends inside a block and a tile
    ([(128, [128, 129, 128])], 8, 8, 128),            # nothing of their own
    ([(256, [300] * 5)], 7, 1, 64),                   # seven heads a group: 126 rows a tile
    ([(400, [401 + 7 * i for i in range(40)])], 6, 2, 128),   # three heads a group
    ([(2000, [2001 + i for i in range(33)])], 16, 1, 64),     # several row tiles, sixteen heads
    ([(2048, [2100 + 13 * i for i in range(70)])], 32, 8, 128),
    ([(4096, [4100 + i for i in range(130)])], 8, 2, 128),    # three pairs of row tiles
    ([(300, [500, 0, 310]), (0, [7, 90]), (5000, [5000, 6100]), (33, [33])], 8, 2, 128),
    ([(640, [700, 100, 0, 16, 641, 640, 639, 624])], 4, 2, 64),   # shorter than the prefix
    ([(100 + 40 * g, [200 + 40 * g, 150 + 40 * g]) for g in range(45)], 4, 2, 64),  # many groups
    ([(20000, [20010, 20500])], 4, 1, 128),           # one unit over all CTAs
    ([(64, [65])] * 3, 12, 12, 64),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("shared", [True, False])
def test_decode(fa, case, shared):
    groups, H, Hkv, d = CASES[case]
    x = Batch(groups, H, Hkv, d, seed=case, shared=shared)
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)
    # bounds that are loose, and no log-sum-exp
    wide = x.table.shape[1] * 16
    again, none = fa.fa_decode_paged_prefix(**x.args(max_prefix_len=min(wide, x.max_pre + 500),
                                                     max_own_len=min(wide, x.max_own + 900)),
                                            want_lse=False)
    assert_device_clean()
    assert none is None
    x.check(again, None, what="loose bounds")


@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_scales_and_equal_rows(fa, scale):
    """Flat and sharp softmaxes; the ordinary call on the same table is as near."""
    x = Batch([(1500, [1501 + 50 * i for i in range(20)])], 8, 2, 128, seed=3)
    out, lse = fa.fa_decode_paged_prefix(**x.args(), scale=scale)
    assert_device_clean()
    G = 4
    for b in range(20):
        k, v = x.rows(x.kp, b), x.rows(x.vp, b)
        for h in range(2):
            q = x.q[b, h * G:h * G + G].double()
            want, wl, tol = ref.forward(q, k[:, h], v[:, h], 0, 0, first=x.ctx[b], scale=scale)
            # scores of 1.0 * |q||k| reach 2^8: fp32 holds them to 2^-16, and a weight
            # follows by as much of itself, as o and the sums do
            far = 2.0 ** -15 * (1 if scale < 1 else 4)
            size = torch_mod().softmax(q @ k[:, h].T * scale, 1) @ v[:, h].abs()
            ref.assert_within(out[b, h * G:h * G + G], want, tol + 2 * far * size)
            assert (lse[b, h * G:h * G + G].double() - wl).abs().max() <= 1e-3


def test_many_rows_deep_prefix(fa):
    """A batch whose products bound the call, checked on some of its sequences."""
    x = Batch([(6000, [6001 + (i * 37) % 400 for i in range(256)])], 32, 8, 128, seed=4)
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse, only=[0, 1, 31, 32, 63, 64, 100, 255])


STRETCHES = [  # groups (prefix, contexts), H, Hkv, d
    ([(2500, [2501 + i for i in range(70)])], 32, 8, 128),    # two pairs of row tiles, twenty key tiles
    ([(2500, [2600] * 40), (1300, [1400] * 35), (130, [150] * 3)], 32, 8, 128),  # unlike pairs
    ([(200 + 40 * g, [260 + 40 * g] * 2) for g in range(33)], 16, 8, 64),        # more than 32 groups
    ([(400 + 70 * g, [440 + 70 * g] * 2) for g in range(24)], 8, 8, 128),        # more pairs than teams
    ([(700, [720] * 3), (300, [310] * 2)], 160, 160, 64),     # more KV heads than CTAs
    ([(1000, [1100] * 9), (260, [300])], 304, 304, 128),
]


@pytest.mark.parametrize("case", range(len(STRETCHES)))
def test_stretches_of_the_work(fa, case):
    """Work that CTAs share out in stretches: ends inside a pair of row tiles, at
    its end and behind it, and KV heads in rounds."""
    groups, H, Hkv, d = STRETCHES[case]
    x = Batch(groups, H, Hkv, d, seed=20 + case)
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    n = len(x.ctx)
    x.check(out, lse, only=sorted({0, 1, 2, n // 3, n // 2, n - 2, n - 1}))
    # the same batch over its own keys alone: each result is off by half a step of
    # its own and half a step of each weight, 2^-8 of sum p |v| <= max |v| each
    few, _ = fa.fa_decode_paged_prefix(**x.args(
        cu_groups=dev(np.zeros(1, np.int32)), prefix_lens=dev(np.zeros(0, np.int32)),
        max_own_len=max(x.ctx)))
    assert_device_clean()
    assert (out.float() - few.float()).abs().max() <= 2.0 ** -6 * x.vp.float().abs().max()


def test_repeated_calls_give_the_same_bits(fa):
    torch = torch_mod()
    x = Batch([(3000, [3010] * 20), (700, [900] * 13)], 16, 4, 128, seed=5)
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(33, 16, 4, 128, x.max_pre, x.max_own))
    first = fa.fa_decode_paged_prefix(**x.args(), workspace=ws)
    for _ in range(5):
        ws[256:].random_(0, 255)   # whatever it held before
        again = fa.fa_decode_paged_prefix(**x.args(), workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert fa.fa_last_device_status(ws) == 0
    assert_device_clean()


@pytest.mark.parametrize("shared", [True, False])
def test_stale_and_foreign_values(fa, shared):
    """NaN in free blocks, in slots past a context and in another group's keys
    reaches nothing; in shared keys it stays in its group."""
    torch = torch_mod()
    x = Batch([(200, [210, 230, 199]), (500, [520, 501]), (90, [100])], 8, 2, 64, seed=6, shared=shared)
    used = np.zeros(x.kp.shape[0] * 16, dtype=bool)
    for b, c in enumerate(x.ctx):
        for j in range(c):
            used[x.table[b, j // 16] * 16 + j % 16] = True
    for pool in (x.kp, x.vp):
        pool.view(-1, 2, 64)[dev(~used)] = math.nan
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)
    x.vp[int(x.table[3, 2]), 5] = math.nan    # a shared key of the second group
    x.kp[int(x.table[3, 3]), 1] = math.inf
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert not torch.isfinite(out[3:5]).any()
    x.check(out, lse, only=[0, 1, 2, 5])


@pytest.mark.parametrize("shared", [True, False])
def test_nan_query(fa, shared):
    torch = torch_mod()
    x = Batch([(300, [320] * 6)], 8, 2, 128, seed=7, shared=shared)
    x.q[2, 3, 17] = math.nan
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert torch.isnan(out[2, 3]).all() and torch.isnan(lse[2, 3])
    x.q[2, 3, 17] = 0
    ok = [0, 1, 3, 4, 5]
    x.check(out, lse, only=ok)
    assert torch.isfinite(out[2, [0, 1, 2, 4, 5, 6, 7]]).all()
    assert_device_clean()


@pytest.mark.parametrize("shared", [True, False])
def test_padded_batch_and_no_groups(fa, shared):
    """Idle slots with tables of nothing, a batch behind its groups, and no
    groups at all."""
    torch = torch_mod()
    x = Batch([(400, [450, 420]), (0, [30, 60])], 8, 2, 64, seed=8, shared=shared)
    x.cu, x.pre = x.cu[:2], x.pre[:1]          # the last two sequences are in no group
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    alone, l1 = fa.fa_decode_paged_prefix(**x.args(
        cu_groups=torch.zeros(1, dtype=torch.int32, device="cuda"), prefix_lens=none,
        max_prefix_len=0, max_own_len=450))
    assert_device_clean()
    x.check(alone, l1)
    x.ctx = [450, 0, 0, 60]
    x.table[1:3] = -1
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    assert not out[1:3].any() and (lse[1:3] == -math.inf).all()
    x.check(out, lse)


@pytest.mark.parametrize("shared", [True, False])
def test_bad_data_is_reported(fa, shared):
    x = Batch([(300, [320, 350]), (100, [120, 130])], 8, 2, 64, seed=9, shared=shared)
    good, gl = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()

    def run(**new):
        ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(4, 8, 2, 64, x.max_pre + 20, 400))
        out, lse = fa.fa_decode_paged_prefix(**x.args(**new), workspace=ws)
        torch_mod().cuda.synchronize()
        st = fa.fa_last_device_status(ws)
        assert fa.fa_device_status() == st
        again, _ = fa.fa_decode_paged_prefix(**x.args(), workspace=ws)   # the workspace recovers
        assert torch_mod().equal(again, good) and fa.fa_last_device_status(ws) == 0
        assert_device_clean()
        return out, lse, st
    i32 = lambda *v: dev(np.int32(v))  # noqa: E731
    out, lse, st = run(ctx_lens=i32(320, -1, 120, 130))
    assert st == fa.FA_DEV_BAD_CTX and not out[1].any() and (lse[1] == -math.inf).all()
    x.check(out, lse, only=[0, 2, 3])
    out, lse, st = run(ctx_lens=i32(320, 350, 120, 200))      # more than max_own_len keys of its own
    assert st == fa.FA_DEV_BAD_CTX and not out[3].any()
    x.check(out, lse, only=[0, 1, 2])
    out, lse, st = run(prefix_lens=i32(x.max_pre + 1, 100))   # beyond max_prefix_len
    assert st == fa.FA_DEV_BAD_CTX and not out[:2].any()
    x.check(out, lse, only=[2, 3])
    out, lse, st = run(cu_groups=i32(0, 2, 5))                # a group outside the batch
    assert st & fa.FA_DEV_BAD_SEQLEN
    x.check(out, lse, only=[0, 1])
    out, lse, st = run(cu_groups=i32(-1, 2, 4), max_own_len=350)
    assert st == fa.FA_DEV_BAD_SEQLEN
    x.check(out, lse)                                         # the first group on its own
    out, lse, st = run(cu_groups=i32(0, 3, 2), max_own_len=352)
    assert st == fa.FA_DEV_BAD_SEQLEN
    x.check(out, lse, only=[0, 1, 3])
    bad = x.table.copy()
    bad[0, 4] = x.kp.shape[0]                                 # a shared block outside the pool
    out, lse, st = run(block_table=dev(bad))
    assert st == fa.FA_DEV_BAD_BLOCK
    x.check(out, lse, only=[2, 3])
    bad = x.table.copy()
    bad[3, 7] = -5                                            # an own one
    out, lse, st = run(block_table=dev(bad))
    assert st == fa.FA_DEV_BAD_BLOCK
    x.check(out, lse, only=[0, 1, 2])


def test_workspace_serves_smaller_calls(fa):
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(64, 8, 2, 128, 9000, 2000))
    for i, groups in enumerate(([(9000, [9001] * 2)], [(500, [2500] * 64)], [(9000, [11000])],
                                [(130, [131] * 64)], [(0, [2000] * 3), (8999, [9100] * 5)])):
        x = Batch(groups, 8, 2, 128, seed=20 + i, shared=False)
        out, lse = fa.fa_decode_paged_prefix(**x.args(), workspace=ws)
        x.check(out, lse, only=[0, len(x.ctx) - 1])
    assert_device_clean()


def test_refusals(fa):
    torch = torch_mod()
    x = Batch([(64, [70, 80])], 8, 2, 64, seed=10, shared=False)
    for new in (dict(q=x.q[:, :, :32]), dict(cu_groups=dev(np.int32([0]))), dict(q=x.q.float()),
                dict(prefix_lens=dev(np.int64([64]))), dict(ctx_lens=dev(np.int32([70]))),
                dict(cu_groups=dev(x.cu).cpu()), dict(q=x.q.transpose(0, 1)), dict(v_pool=x.vp[1:]),
                dict(block_table=dev(x.table)[0]), dict(workspace=torch.zeros(4, device="cuda")),
                dict(out=torch.zeros(2, 8, 64, device="cuda"))):
        with pytest.raises(ValueError):
            fa.fa_decode_paged_prefix(**x.args(**new))
    for new in (dict(max_prefix_len=-1), dict(max_own_len=10000), dict(scale=-1.0),
                dict(workspace=fa.new_workspace(512))):
        with pytest.raises(fa.FaError):
            fa.fa_decode_paged_prefix(**x.args(**new))
    q = x.q[:0]
    out, lse = fa.fa_decode_paged_prefix(**x.args(
        q=q, block_table=dev(x.table[:0]), ctx_lens=dev(np.int32([])), cu_groups=dev(np.int32([0])),
        prefix_lens=dev(np.int32([]))))
    assert out.shape == q.shape and lse.shape == (0, 8)


def test_streams_and_two_calls_at_once(fa):
    """Two calls on two streams with workspaces of their own."""
    torch = torch_mod()
    xs = [Batch([(2500, [2600] * 24)], 8, 2, 128, seed=30), Batch([(700, [900] * 9)], 8, 2, 128, seed=31)]
    streams = [torch.cuda.Stream() for _ in xs]
    args = [x.args() for x in xs]
    ws = [fa.new_workspace(fa.fa_decode_prefix_workspace_size(24, 8, 2, 128, x.max_pre, 200)) for x in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [fa.fa_decode_paged_prefix(**a, workspace=w, stream=s)
               for a, w, s in zip(args, ws, streams)]
    torch.cuda.synchronize()
    for x, (out, lse) in zip(xs, got):
        x.check(out, lse, only=[0, len(x.ctx) - 1])
    assert_device_clean()


@pytest.mark.parametrize("most", [1000, 20000])   # every key as an own one, and shared
def test_graph_replay_with_new_groups(fa, most):
    """A captured call replayed on other groups, lengths, queries and blocks
    inside its bounds; two graphs share a workspace one after the other."""
    torch = torch_mod()
    shapes = [[(900, [950] * 6), (0, [40] * 2)], [(100, [150]), (700, [701] * 4 + [800, 0, 650])],
              [(16, [60, 17]), (1000, [1001] * 6)]]
    xs = [Batch(s, 8, 2, 64, seed=40 + i, shared=False) for i, s in enumerate(shapes)]
    blocks = max(x.kp.shape[0] for x in xs)
    width = max([(most + 15) // 16] + [x.table.shape[1] for x in xs])
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    kp, vp, q = z(blocks, 16, 2, 64), z(blocks, 16, 2, 64), z(8, 8, 64)
    table, ctx, cu, pre = (z(8, width, t=torch.int32), z(8, t=torch.int32), z(3, t=torch.int32),
                           z(2, t=torch.int32))
    out, lse = torch.empty_like(q), z(8, 8, t=torch.float32)
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(8, 8, 2, 64, most, 100))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            fa.fa_decode_paged_prefix(q, kp, vp, table, ctx, cu, pre, most, 100, out=out, lse=lse,
                                      workspace=ws)
    for turn, x in enumerate(xs * 2):
        kp[:x.kp.shape[0]] = x.kp
        vp[:x.vp.shape[0]] = x.vp
        table.fill_(-1)
        table[:, :x.table.shape[1]] = dev(x.table)
        q.copy_(x.q), ctx.copy_(dev(np.int32(x.ctx))), cu.copy_(dev(x.cu)), pre.copy_(dev(x.pre))
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        x.check(out, lse, what=f"replay {turn}")
    assert_device_clean()


def test_far_blocks(fa):
    """A pool of more than 2^31 values."""
    torch = torch_mod()
    Hkv, d = 64, 128
    blocks = (1 << 31) // (16 * Hkv * d) + 8
    x = Batch([(64, [70, 66])], 64, Hkv, d, seed=11)
    kp, vp = (torch.zeros((blocks, 16, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    shift = blocks - x.kp.shape[0]
    kp[shift:], vp[shift:] = x.kp, x.vp
    table = np.where(x.table >= 0, x.table + shift, -1).astype(np.int32)
    out, lse = fa.fa_decode_paged_prefix(**x.args(k_pool=kp, v_pool=vp, block_table=dev(table)))
    assert_device_clean()
    x.check(out, lse)


@pytest.mark.parametrize("most", [300, 20000])   # every key as an own one, and shared
def test_serving_run(fa, most):
    """One prompt written once, then tokens of several samples of it: each step
    writes rotated keys and reads the shared blocks through
    fa_decode_paged_prefix; every step against attention in 64 bits over rotated
    keys as they were projected."""
    torch = torch_mod()
    rng = np.random.default_rng(12)
    H, Hkv, d, n, prompt, steps = 8, 2, 128, 9, 300, 4
    freq = rr.frequencies(d)
    f = dev(freq)
    whole = prompt // 16
    own = (prompt + steps + 15) // 16 - whole
    perm = rng.permutation(whole + n * own + 2)
    table = np.int32([[*perm[:whole], *perm[whole + i * own: whole + (i + 1) * own]] for i in range(n)])
    table = np.pad(table, ((0, 0), (0, max(0, most // 16 - table.shape[1]))), constant_values=-1)
    pools = [torch.zeros((len(perm), 16, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    bf = lambda a: dev(a).to(torch.bfloat16)  # noqa: E731
    k0, v0 = (cr.bf16(rng, prompt, Hkv, d) for _ in "kv")
    # the prompt through the first sample's table; the part block is copied for the others
    fa.fa_cache_append_rope(None, bf(k0), bf(v0), f, *pools, dev(table[:1]), dev(np.int32([prompt])),
                            dev(np.int32([0, prompt])), prompt)
    for pool in pools:
        pool[dev(table[1:, whole].astype(np.int64))] = pool[int(table[0, whole])].clone()
    keys = [[k0] for _ in range(n)]
    vals = [[v0] for _ in range(n)]
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(n, H, Hkv, d, most, steps))
    for step in range(1, steps + 1):
        q, k, v = (cr.bf16(rng, n, h, d) for h in (H, Hkv, Hkv))
        ctx = dev(np.int32([prompt + step] * n))
        qr = fa.fa_cache_append_rope(bf(q), bf(k), bf(v), f, *pools, dev(table), ctx,
                                     dev(np.arange(n + 1, dtype=np.int32)), 1)
        out, lse = fa.fa_decode_paged_prefix(qr, *pools, dev(table), ctx, dev(np.int32([0, n])),
                                             dev(np.int32([prompt])), most, steps, workspace=ws)
        for b in range(n):
            keys[b].append(k[b:b + 1]), vals[b].append(v[b:b + 1])
            kk = rr.rotate(np.concatenate(keys[b]), np.arange(prompt + step), freq)
            vv = np.concatenate(vals[b]).astype(np.float64)
            qq = rr.rotate(q[b:b + 1], [prompt + step - 1], freq)[0]
            for h in range(H):
                # q and k rounded once each: a score moves by 2 * 2^-8 sum |q||k| / sqrt(d) at
                # most, and a weight by that of itself
                x = kk[:, h // 4] @ qq[h] / math.sqrt(d)
                move = (2 * rr.U * (np.abs(kk[:, h // 4]) @ np.abs(qq[h])) / math.sqrt(d)).max() * 1.05
                w = np.exp(x - x.max())
                w /= w.sum()
                want, size = w @ vv[:, h // 4], w @ np.abs(vv[:, h // 4])
                tol = (np.expm1(2 * move) + 3 * rr.U) * size + rr.U * np.abs(want)
                got = out[b, h].double().cpu().numpy()
                assert (np.abs(got - want) <= tol).all(), (step, b, h)
    assert_device_clean()


def reaching(x):
    """The batch's table made as wide as its longest prefix, which the call wants
    although none of its sequences may be as long."""
    more = (x.max_pre + 15) // 16 - x.table.shape[1]
    x.table = np.pad(x.table, ((0, 0), (0, max(0, more))), constant_values=-1)
    return x


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("rest", [-1, "stale"])
@pytest.mark.parametrize("groups", [
    [(400, [0, 450, 420]), (90, [100, 0])],                # a finished sequence comes first
    [(1001, [100, 0, 1040, 1002])],                        # ... or one of few keys
    [(700, [0] * 40 + [710, 30, 705]), (0, [50])],         # the 41st has them all
    [(2048, [2047, 2030, 2048, 2100])],                    # short by one key
    [(2500, [300, 1234, 0, 1233]), (640, [640])],          # none has them all
    [(300, [0, 0]), (64, [70])],                           # nobody is there
])
def test_rows_hold_the_blocks_of_their_keys_alone(fa, groups, rest, shared):
    """A group's shared blocks are found whichever of its sequences has them: a
    row holds nothing, or old ids, behind its own keys."""
    x = reaching(Batch(groups, 8, 2, 128, seed=50, shared=shared))
    for b, c in enumerate(x.ctx):
        x.table[b, (c + 15) // 16:] = -1 if rest == -1 else x.table[b, 0] if c else b
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)
    assert not out[[b for b, c in enumerate(x.ctx) if c == 0]].any()


@pytest.mark.parametrize("groups,H,Hkv,d", [
    ([(640, [700, 100, 0, 16, 641, 640, 639, 624])], 4, 2, 64),    # one row tile: both streams
    ([(2000, [1500, 2010, 700] + [2001] * 60), (320, [330, 15])], 32, 8, 128),   # 2080 rows
    ([(1000, [1010] * 50 + [129, 990, 500] + [1002] * 20)], 32, 8, 128),   # 2336 rows
    ([(512, [515] * 140 + [200, 333])], 32, 8, 64),                # 4544 rows
])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("shared", [True, False])
def test_values_behind_a_short_sequence(fa, groups, H, Hkv, d, value, shared):
    """A sequence that ends inside the shared keys meets nothing of those behind
    its own, whatever they hold; those that see them do."""
    torch = torch_mod()
    x = Batch(groups, H, Hkv, d, seed=60, shared=shared)
    a, e = int(x.cu[0]), int(x.cu[1])
    long = [b for b in range(a, e) if x.ctx[b] >= groups[0][0]]
    short = [b for b in range(len(x.ctx)) if b not in long]
    last = max(x.ctx[b] for b in short if b < e)
    x.vp[int(x.table[0, last // 16]), last % 16] = value   # the first key that no short one sees
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse, only=short)
    assert not torch.isfinite(out[long]).any() and torch.isfinite(lse[long]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared", [True, False])
def test_slots_that_nobody_wrote(fa, d, shared):
    """All sequences of a group shorter than its prefix: its other slots are free
    ones and hold NaN."""
    x = reaching(Batch([(900, [500, 0, 507, 64]), (300, [17])], 8, 2, d, seed=61, shared=shared))
    used = np.zeros(x.kp.shape[0] * 16, dtype=bool)
    for b, c in enumerate(x.ctx):
        for j in range(c):
            used[x.table[b, j // 16] * 16 + j % 16] = True
    for pool in (x.kp, x.vp):
        pool.view(-1, 2, d)[dev(~used)] = math.nan
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)


@pytest.mark.parametrize("shared", [True, False])
def test_short_sequences_keep_what_is_theirs(fa, shared):
    """Infinite and NaN values that a short sequence does see, and a query of its
    that holds a NaN, come through as they do for any other."""
    torch = torch_mod()
    x = Batch([(800, [810, 300, 400, 200])], 8, 2, 128, seed=62, shared=shared)
    x.vp[int(x.table[0, 20]), 3] = math.nan      # key 323: sequences 0 and 2 see it
    x.q[3, 5, 9] = math.nan
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    assert torch.isnan(out[[0, 2]]).all() and torch.isfinite(lse[[0, 2]]).all()
    x.check(out, lse, only=[1])
    assert torch.isnan(out[3, 5]).all() and torch.isnan(lse[3, 5])
    assert torch.isfinite(out[3, [0, 1, 2, 3, 4, 6, 7]]).all()


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("cu,kept", [
    ([0, 4, 2, 6], [0]), ([0, 4, 2, 4], [0]), ([0, 6, 5, 3, 6], [0]), ([0, 2, 1, 4, 3, 6], [0]),
    ([0, 3, 1, 3, 6], [0, 3]), ([2, 0, 4, 4, 6], [1, 2, 3]),
])
def test_groups_that_go_back(fa, cu, kept, shared):
    """cu_groups that falls: a group that would begin inside an earlier one is
    passed over as the one of negative size is, and its sequences read their keys
    as own ones."""
    x = Batch([(700, [720, 705, 710, 800, 777, 701])], 8, 2, 128, seed=70, shared=shared)
    groups = len(cu) - 1
    args = x.args(cu_groups=dev(np.int32(cu)), max_own_len=800,
                  prefix_lens=dev(np.int32([700 - 16 * g for g in range(groups)])))
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(6, 8, 2, 128, x.max_pre, 800))
    first = fa.fa_decode_paged_prefix(**args, workspace=ws)
    torch_mod().cuda.synchronize()
    assert fa.fa_last_device_status(ws) == fa.FA_DEV_BAD_SEQLEN
    x.check(*first)
    for _ in range(3):
        again = fa.fa_decode_paged_prefix(**args, workspace=ws)
        assert all(torch_mod().equal(p, q) for p, q in zip(again, first))
    # the groups that stand, alone in the call
    for g in kept:
        x.check(*fa.fa_decode_paged_prefix(**{**args, "cu_groups": dev(np.int32(cu[g:g + 2])),
                                              "prefix_lens": args["prefix_lens"][g:g + 1]}, workspace=ws))
        assert fa.fa_last_device_status(ws) == 0
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_SEQLEN


def test_groups_that_go_back_far_down(fa):
    """The same among more than 32 groups, so that the walk over them has steps."""
    n = 80
    x = Batch([(320, [330 + b for b in range(n)])], 4, 2, 64, seed=71)
    cu = list(range(0, 60)) + [50] + list(range(51, 70))   # group 59 falls, 60 to 68 begin too early
    args = x.args(cu_groups=dev(np.int32(cu)), prefix_lens=dev(np.int32([320] * (len(cu) - 1))),
                  max_own_len=410)
    ws = fa.new_workspace(fa.fa_decode_prefix_workspace_size(n, 4, 2, 64, x.max_pre, 410))
    out, lse = fa.fa_decode_paged_prefix(**args, workspace=ws)
    torch_mod().cuda.synchronize()
    assert fa.fa_last_device_status(ws) == fa.FA_DEV_BAD_SEQLEN
    assert fa.fa_device_status(clear=True) == fa.FA_DEV_BAD_SEQLEN
    x.check(out, lse)


@pytest.mark.parametrize("shared", [True, False])
def test_more_groups_than_sequences(fa, shared):
    """An array of groups of a fixed size, empty ones behind and between."""
    x = Batch([(500, [520, 510]), (0, []), (64, [100]), *[(0, [])] * 60], 8, 2, 64, seed=90, shared=shared)
    out, lse = fa.fa_decode_paged_prefix(**x.args())
    assert_device_clean()
    x.check(out, lse)


@pytest.mark.parametrize("members,idle,G", [(48, 16, 4), (100, 28, 4), (50, 14, 8)])
def test_idle_slots_leave_the_plan_alone(fa, members, idle, G):
    """Finished slots at a group's end have nothing to read and nothing to share:
    the work is shared out as if they were in no group, bit for bit."""
    torch = torch_mod()
    x = Batch([(8192, [8192 + 37 + (i * 131) % 900 for i in range(members)] + [0] * idle)], 8 * G, 8,
              128, seed=80)
    inside = fa.fa_decode_paged_prefix(**x.args())
    outside = fa.fa_decode_paged_prefix(**x.args(cu_groups=dev(np.int32([0, members]))))
    assert_device_clean()
    assert all(torch.equal(a, b) for a, b in zip(inside, outside))
    x.check(*inside, only=[0, members - 1, members])
