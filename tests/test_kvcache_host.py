"""Host-side checks of the 8-bit cache's calls (no GPU): exported and bound,
arguments refused before any launch, and the tests' NumPy twin against plain
statements."""
import ctypes
import os
import re

import numpy as np
import pytest

import cache_reference as cr
from exact_attention_33_gb300 import workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
P_BAD = ctypes.c_void_p(0x10008)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa
    return fa.load_library()


def test_header_is_exported_and_bound(lib):
    import exact_attention_33_gb300 as fa
    text = open(os.path.join(ROOT, "include", "fa_kvcache.h")).read()
    names = set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"fa_cache_append_fp8", "fa_decode_paged_fp8", "fa_fwd_paged_fp8"}
    for name in names:
        assert hasattr(lib, name) and callable(getattr(fa, name)) and name in fa.__all__, name


def test_append_refusals(lib):
    def call(k=P, ks=256, vs=256, pool=P, scale=P, table=P, width=4, cu=P, batch=2, total=4,
             new=4, Hkv=2, d=128, bs=16, nb=8):
        return lib.fa_cache_append_fp8(k, P, ks, vs, pool, P, scale, P, table, width, P, cu, batch,
                                       total, new, Hkv, d, bs, nb, NULL)
    assert call(k=NULL) == -1 and call(pool=NULL) == -1 and call(scale=NULL) == -1
    assert call(k=P_BAD) == -1 and call(pool=P_BAD) == -1 and call(cu=NULL) == -1
    assert call(ks=255) == -1 and call(vs=260) == -1 and call(ks=0) == -1
    assert call(Hkv=0) == -1 and call(nb=0) == -1 and call(width=0) == -1 and call(batch=-1) == -1
    assert call(d=96) == -2 and call(bs=32) == -2 and call(batch=70000) == -2
    assert call(nb=1 << 28) == -2
    assert call(batch=0) == 0 and call(total=0) == 0 and call(new=0) == 0


def test_decode_refusals(lib):
    def call(q=P, scale_ptr=P, max_ctx=64, batch=2, H=8, d=128, bs=16, window=0, sinks=0, ws=P,
             size=1 << 20, scale=0.1):
        return lib.fa_decode_paged_fp8(q, P, P, scale_ptr, P, P, 4, P, max_ctx, batch, H, 2, d, bs,
                                       8, scale, window, sinks, P, NULL, ws, size, NULL)
    assert call(q=NULL) == -1 and call(q=P_BAD) == -1 and call(scale_ptr=NULL) == -1
    assert call(max_ctx=65) == -1 and call(H=7) == -1 and call(scale=0.0) == -1
    assert call(window=-1) == -1 and call(sinks=2) == -1 and call(window=4, sinks=-1) == -1
    assert call(H=64) == -2 and call(d=80) == -2 and call(bs=8) == -2
    assert call(ws=NULL) == -4 and call(size=64) == -4 and call(batch=0) == 0


def test_chunk_refusals(lib):
    def call(q=P, scale_ptr=P, cu=P, total=4, max_ctx=64, H=8, d=128, window=0, sinks=0):
        return lib.fa_fwd_paged_fp8(q, P, P, scale_ptr, P, P, 4, P, cu, 2, total, 4, max_ctx, H, 2, d,
                                    16, 8, 0.1, window, sinks, P, NULL, NULL)
    assert call(q=NULL) == -1 and call(q=P_BAD) == -1 and call(scale_ptr=NULL) == -1
    assert call(cu=NULL) == -1 and call(max_ctx=65) == -1 and call(H=7) == -1
    assert call(window=-2) == -1 and call(sinks=1) == -1 and call(d=96) == -2 and call(total=0) == 0


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    import exact_attention_33_gb300 as fa
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.uint8)
    scale = torch.ones((2, 2))
    i = torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_decode_paged_fp8(q, pool, pool, scale, scale, i[None], i, 1)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_fp8(q, pool, pool, scale, scale, i[None], i, i, 1, 1)
    with pytest.raises(ValueError):
        fa.fa_cache_append_fp8(q, q, pool, pool, scale, scale, i[None], i, i, 1)


def test_twin_scales_are_the_smallest_powers_of_two():
    for amax in (0.0, 1e-40, 3.0, 7.0, 7.0000005, 448.0, 448.1, 1e38):
        s = float(cr.need_scale(amax))
        assert amax <= 448 * s and np.log2(s) == np.floor(np.log2(s)) and s >= 2.0 ** -100
        assert s == 2.0 ** -100 or amax > 448 * s / 2


def test_twin_rounds_once():
    """A block written at once is within half a step of its values, and one
    filled token by token within one half step more below e4m3's normal range."""
    rng = np.random.default_rng(0)
    x = cr.bf16(rng, 16, 1, 64) * np.exp2(rng.integers(-6, 3, (16, 1, 1))).astype(np.float32)
    whole, ws = np.zeros((1, 16, 1, 64), np.uint8), np.zeros((1, 1), np.float32)
    cr.append(x, whole, ws, [[0]], [16], [16])
    step = np.maximum(np.abs(x) * 2.0 ** -4, float(ws[0, 0]) * 2.0 ** -10)
    assert (np.abs(cr.real(whole, ws)[0] - x) <= step).all()
    by_one, s = np.zeros_like(whole), np.zeros_like(ws)
    for n in range(1, 17):
        cr.append(x[n - 1:n], by_one, s, [[0]], [n], [1])
    assert s[0, 0] == ws[0, 0]
    off = np.abs(cr.real(by_one, s) - cr.real(whole, ws))
    assert (off <= float(ws[0, 0]) * 2.0 ** -9).all()
