"""Host-side checks of decoding over shared prefixes (no GPU): exported and
bound, arguments refused before any launch, workspace sizes."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
P_BAD = ctypes.c_void_p(0x10008)
P_ODD = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa
    return fa.load_library()


def test_header_is_exported_and_bound(lib):
    import exact_attention_33_gb300 as fa
    text = open(os.path.join(ROOT, "include", "fa_prefix.h")).read()
    names = set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    names.discard("fa_decode_prefix_workspace_size()")
    assert names == {"fa_decode_paged_prefix", "fa_decode_prefix_workspace_size"}
    for name in names:
        assert hasattr(lib, name) and callable(getattr(fa, name)) and name in fa.__all__, name


def test_refusals(lib):
    def call(q=P, kp=P, table=P, width=8, ctx=P, cu=P, pre=P, groups=1, mp=64, mo=64, batch=2, H=8,
             Hkv=2, d=128, bs=16, nb=8, scale=0.1, out=P, lse=NULL, ws=P, size=1 << 30):
        return lib.fa_decode_paged_prefix(q, kp, P, table, width, ctx, cu, pre, groups, mp, mo, batch,
                                          H, Hkv, d, bs, nb, scale, out, lse, ws, size, NULL)
    assert call(batch=0) == 0 and call(batch=0, groups=0, cu=NULL, pre=NULL) == 0
    for name in ("q", "kp", "table", "ctx", "cu", "pre", "out"):
        assert call(**{name: NULL}) == -1, name
    for name in ("q", "kp", "out"):
        assert call(**{name: P_BAD}) == -1, name
    for name in ("table", "ctx", "cu", "pre", "lse"):
        assert call(**{name: P_ODD}) == -1, name
    assert call(groups=-1) == -1 and call(batch=-1) == -1 and call(mp=-1) == -1 and call(mo=-1) == -1
    assert call(mp=129) == -1 and call(mo=129) == -1 and call(H=7) == -1 and call(nb=0) == -1
    assert call(width=0) == -1 and call(scale=0.0) == -1 and call(scale=float("nan")) == -1
    assert call(d=96) == -2 and call(bs=32) == -2 and call(H=34) == -2 and call(batch=70000) == -2
    assert call(nb=1 << 28) == -2
    assert call(width=1 << 27, mp=1 << 30, mo=1 << 30) == -2   # positions past 32 bits
    assert call(width=1 << 26, mp=1 << 29, batch=60000, groups=60000) == -2
    assert call(ws=NULL) == -4 and call(ws=P_BAD) == -4 and call(size=256) == -4


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    import exact_attention_33_gb300 as fa
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_decode_paged_prefix(q, pool, pool, i[None], i, torch.zeros(2, dtype=torch.int32), i, 1, 1)


def test_workspace_sizes_rise(lib):
    import exact_attention_33_gb300 as fa

    def rises(sizes):
        return all(a <= b for a, b in zip(sizes, sizes[1:]))
    lengths = sorted({0, 1, 15, *range(16, 2200, 90), 4096, 20000, 1 << 20})
    for H, Hkv, d in ((32, 8, 128), (8, 8, 64), (16, 1, 128)):
        at = lambda b, p, o: fa.fa_decode_prefix_workspace_size(b, H, Hkv, d, p, o)  # noqa: E731
        for n in (0, 100, 5000):
            assert rises([at(7, p, n) for p in lengths]) and rises([at(7, n, o) for o in lengths])
            assert rises([at(b, n, 300) for b in range(1, 300, 7)])
    size = fa.fa_decode_prefix_workspace_size
    assert size(1, 8, 2, 96, 1, 1) == 0 and size(1, 7, 2, 64, 1, 1) == 0 and size(-1, 8, 2, 64, 1, 1) == 0
    assert size(1, 8, 2, 64, -1, 1) == 0 and size(1, 8, 2, 64, 1 << 30, 1 << 30) == 0
    assert size(1, 8, 2, 64, 1, 1, block_size=32) == 0


def test_more_groups_than_sequences_are_taken(lib):
    """Empty groups are no work: up to 65535 of them, whatever the batch, as long as
    the sequences cannot make too much of it (-4: the call came to its workspace)."""
    def call(groups, batch=2, mp=64, width=8, Hkv=2):
        return lib.fa_decode_paged_prefix(P, P, P, P, width, P, P, P, groups, mp, 64, batch, 4 * Hkv,
                                          Hkv, 128, 16, 8, 0.1, P, NULL, NULL, 0, NULL)
    assert call(3) == -4 and call(2) == -4 and call(65535) == -4
    assert call(65536) == -2 and call((1 << 31) - 1) == -2
    # 4096 sequences, 64 Ki keys shared: 8192 slots for groups are no more work than 4096
    big = dict(batch=4096, mp=1 << 16, width=1 << 12, Hkv=8)
    assert call(1, **big) == -4 and call(4096, **big) == -4 and call(8192, **big) == -4
    assert call(65535, **big) == -4
    # 60000 sequences that may be a group each, over 2^29 keys
    assert call(1, batch=60000, mp=1 << 29, width=1 << 26) == -2
    assert call(60000, batch=60000, mp=1 << 29, width=1 << 26) == -2
