"""Host-side checks of the rotary calls (no GPU): exported and bound, arguments
refused before any launch, the frequencies, and the tests' NumPy twin against
plain statements."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import rope_reference as rr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
P2 = ctypes.c_void_p(0x20000)
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
    text = open(os.path.join(ROOT, "include", "fa_rope.h")).read()
    names = set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"fa_rope", "fa_rope_bwd", "fa_cache_append_rope", "fa_cache_append_rope_fp8"}
    for name in names:
        assert hasattr(lib, name) and callable(getattr(fa, name)) and name in fa.__all__, name


@pytest.mark.parametrize("name", ["fa_rope", "fa_rope_bwd"])
def test_rope_refusals(lib, name):
    def call(q=P, k=P, qs=1024, ks=256, qo=P2, ko=P2, qos=1024, kos=256, freq=P, rot=128, factor=1.0,
             pos=P, n=1, total=4, H=8, Hkv=2, d=128):
        return getattr(lib, name)(q, k, qs, ks, qo, ko, qos, kos, freq, rot, factor, 0, pos, n, total,
                                  H, Hkv, d, NULL)
    assert call(total=0) == 0 and call(total=0, Hkv=0, k=NULL, ko=NULL) == 0
    assert call(total=0, pos=NULL) == 0
    assert call(q=NULL) == -1 and call(k=NULL) == -1 and call(qo=NULL) == -1 and call(ko=NULL) == -1
    assert call(q=P_BAD) == -1 and call(ko=P_BAD) == -1 and call(freq=NULL) == -1
    assert call(freq=ctypes.c_void_p(0x10004)) == -1 and call(pos=ctypes.c_void_p(0x10002)) == -1
    assert call(qs=1023) == -1 and call(qs=1016) == -1 and call(kos=260) == -1 and call(ks=0) == -1
    assert call(qo=P, qos=2048) == -1                      # in place at another stride
    assert call(rot=0) == -1 and call(rot=-16) == -1 and call(rot=144) == -1
    assert call(rot=24) == -2 and call(rot=120) == -2 and call(d=96) == -2
    assert call(factor=0.0) == -1 and call(factor=math.inf) == -1 and call(factor=math.nan) == -1
    assert call(pos=NULL, n=0) == -1 and call(total=-1) == -1 and call(H=0) == -1
    assert call(Hkv=-1) == -1
    assert call(H=70000, qs=70000 * 128, qos=70000 * 128) == -2


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(lib, fp8):
    def call(q=P, k=P, v=P, qs=1024, ks=256, vs=256, qo=P2, qos=1024, freq=P, rot=128, factor=1.0,
             pool=P, scale=P, table=P, width=4, ctx=P, cu=P, batch=2, total=4, new=4, H=8, Hkv=2,
             d=128, bs=16, nb=8):
        scales = (scale, P) if fp8 else ()
        f = lib.fa_cache_append_rope_fp8 if fp8 else lib.fa_cache_append_rope
        return f(q, k, v, qs, ks, vs, qo, qos, freq, rot, factor, 1, pool, P, *scales, table, width,
                 ctx, cu, batch, total, new, H, Hkv, d, bs, nb, NULL)
    for none in (dict(batch=0), dict(total=0), dict(new=0), dict(new=0, q=NULL, qo=NULL, H=0)):
        assert call(**none) == 0, none
    for name in ("k", "v", "pool", "table", "ctx", "cu"):
        assert call(**{name: NULL}) == -1, name
    assert call(q=NULL) == -1 and call(qo=NULL) == -1     # one without the other
    assert call(k=P_BAD) == -1 and call(q=P_BAD) == -1 and call(pool=P_BAD) == -1
    assert call(ks=255) == -1 and call(vs=260) == -1 and call(qos=1000) == -1 and call(H=0) == -1
    assert call(Hkv=0) == -1 and call(nb=0) == -1 and call(width=0) == -1 and call(batch=-1) == -1
    assert call(rot=136) == -1 and call(rot=40) == -2 and call(factor=-1.0) == -1
    assert call(freq=NULL) == -1
    assert call(freq=NULL, rot=0, new=0) == (-1 if fp8 else 0)
    assert call(d=96) == -2 and call(bs=32) == -2 and call(batch=70000) == -2
    assert call(nb=1 << 28) == -2
    if fp8:
        assert call(scale=NULL) == -1 and call(rot=0) == -1


def test_binding_rejects():
    torch = pytest.importorskip("torch")
    import exact_attention_33_gb300 as fa
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    f = torch.ones(32, dtype=torch.float64)
    pool = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_rope(q, q, f)
    with pytest.raises(ValueError):
        fa.fa_rope_bwd(q, None, f)
    with pytest.raises(ValueError):
        fa.fa_cache_append_rope(q, q, q, f, pool, pool, i[None], i, i, 1)
    with pytest.raises(ValueError):
        fa.fa_cache_append_rope_fp8(q, q, q, None, pool, pool, i, i, i[None], i, i, 1)


def test_frequencies():
    pytest.importorskip("torch")
    import exact_attention_33_gb300 as fa

    def get(*a, **k):
        f, factor = fa.fa_rope_frequencies(*a, device="cpu", **k)
        return f.numpy(), factor
    plain, factor = get(64)
    assert factor == 1.0 and np.allclose(plain, rr.frequencies(64), rtol=1e-14)
    slow, _ = get(64, stretch=4.0, method="linear")
    assert np.allclose(slow, plain / 4, rtol=1e-14)
    based, _ = get(64, stretch=4.0, method="base")
    assert based[0] == 1.0 and np.isclose(based[-1], plain[-1] / 4, rtol=1e-12)
    parts, factor = get(128, base=500000.0, stretch=8.0, trained_len=8192)
    whole = rr.frequencies(128, 500000.0)
    turns = 8192 * whole / (2 * np.pi)
    assert np.allclose(parts[turns >= 32], whole[turns >= 32], rtol=1e-12)
    assert np.allclose(parts[turns <= 1], whole[turns <= 1] / 8, rtol=1e-12)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (parts[between] < whole[between]).all()
    assert (parts[between] > whole[between] / 8).all() and np.isclose(factor, 1 + 0.1 * np.log(8.0))
    assert get(64, stretch=1.0)[1] == 1.0
    for bad in (dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=64, base=1.0),
                dict(rot_dim=64, stretch=0.5), dict(rot_dim=64, method="other"),
                dict(rot_dim=64, stretch=2.0, slow_turns=4.0, fast_turns=4.0)):
        with pytest.raises(ValueError):
            fa.fa_rope_frequencies(**bad, device="cpu")


@pytest.mark.parametrize("interleaved", [False, True])
def test_twin(interleaved):
    """Angles add up, lengths stay, scores depend on the distance alone, and the
    gradient's rotation is the transpose: against differences too."""
    rng = np.random.default_rng(0)
    f = rr.frequencies(48)
    x, y = rng.standard_normal((2, 5, 3, 64))
    rot = lambda z, p, **k: rr.rotate(z, np.full(5, p), f, interleaved=interleaved, **k)  # noqa: E731
    assert np.allclose(rot(rot(x, 3), 4), rot(x, 7), atol=1e-12)
    assert np.allclose((rot(x, 9) ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose((rot(x, 109) * rot(y, 102)).sum(-1), (rot(x, 7) * y).sum(-1), atol=1e-11)
    g = rot(y, 6, factor=1.3, back=True)
    assert np.allclose((rot(x, 6, factor=1.3) * y).sum(), (x * g).sum())
    u, h = rng.standard_normal(x.shape), 1e-4
    moved = [(rot(x + t * u, 6, factor=1.3) * y).sum() for t in (h, -h)]
    assert np.isclose((moved[0] - moved[1]) / (2 * h), (u * g).sum(), rtol=1e-9)
    assert (rot(x, 5)[..., 48:] == x[..., 48:]).all()


def test_twin_scales():
    """A rotated key never leaves the range of a scale taken before the rotation."""
    rng = np.random.default_rng(1)
    f = rr.frequencies(64)
    for factor in (1.0, 1.27, 0.5):
        x = rng.standard_normal((200, 1, 64)) * np.exp2(rng.integers(-8, 8, (200, 1, 1)))
        x = x.astype(np.float32).astype(np.float64)
        y = rr.rotate(x, rng.integers(0, 100000, 200), f, factor)
        for a, b in zip(x, y):
            s = rr.need_scale(np.abs(a).max(), rr.grow_of(factor))
            assert np.abs(b).max() <= 448 * s * (1 + 2.0 ** -23)
