"""Host-side checks of the windowed calls (no GPU): the header's calls are
exported and bound, arguments are refused before any launch, and the 64-bit
reference that the GPU tests use agrees with the oracle and with differences."""
import ctypes
import os
import re

import numpy as np
import pytest

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
    text = open(os.path.join(ROOT, "include", "fa_window.h")).read()
    names = set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 8
    for name in names:
        assert hasattr(lib, name) and callable(getattr(fa, name)) and name in fa.__all__, name


def fwd(lib, q=P, B=1, H=2, Hkv=2, N=16, d=64, scale=0.125, window=4, sinks=0):
    return lib.fa_fwd_window(q, P, P, P, NULL, B, H, Hkv, N, d, scale, window, sinks, NULL)


def test_dense_refusals(lib):
    assert fwd(lib, window=0) == -1 and fwd(lib, window=-3) == -1 and fwd(lib, sinks=-1) == -1
    assert fwd(lib, q=NULL) == -1 and fwd(lib, q=P_BAD) == -1 and fwd(lib, H=3) == -1
    assert fwd(lib, d=96) == -2 and fwd(lib, scale=0.0) == -1 and fwd(lib, scale=float("inf")) == -1
    assert fwd(lib, N=0) == 0 and fwd(lib, B=0) == 0


def test_packed_refusals(lib):
    def call(cu=P, seqs=2, window=4, sinks=1, d=64):
        return lib.fa_fwd_varlen_window(P, P, P, P, NULL, cu, seqs, 10, 5, 2, 2, d, 0.1, window,
                                        sinks, NULL)
    assert call(cu=NULL) == -1 and call(window=0) == -1 and call(sinks=-1) == -1
    assert call(seqs=-1) == -1 and call(d=80) == -2 and call(seqs=0) == 0


def test_cached_refusals(lib):
    def decode(window=4, sinks=0, bs=16, ws=P, size=1 << 20, max_ctx=64, H=8, batch=2):
        return lib.fa_decode_paged_window(P, P, P, P, 4, P, max_ctx, batch, H, 2, 128, bs, 8, 0.1,
                                          window, sinks, P, NULL, ws, size, NULL)
    assert decode(window=0) == -1 and decode(sinks=-1) == -1 and decode(max_ctx=65) == -1
    assert decode(bs=32) == -2 and decode(H=64) == -2 and decode(batch=0) == 0
    assert decode(ws=NULL) == -4 and decode(size=16) == -4

    def chunk(window=4, sinks=0, total=4):
        return lib.fa_fwd_paged_window(P, P, P, P, 4, P, P, 2, total, 4, 64, 8, 2, 128, 16, 8, 0.1,
                                       window, sinks, P, NULL, NULL)
    assert chunk(window=0) == -1 and chunk(sinks=-5) == -1 and chunk(total=0) == 0


def test_backward_refusals(lib):
    def call(window=4, sinks=0, ws=P, size=1 << 20, lse=P, N=16):
        return lib.fa_bwd_window(P, P, P, P, lse, P, P, P, P, 1, 2, 2, N, 64, 0.1, window, sinks,
                                 ws, size, NULL)
    assert call(window=0) == -1 and call(sinks=-1) == -1 and call(lse=NULL) == -1
    assert call(ws=NULL) == -4 and call(size=8) == -4 and call(N=0) == 0

    def packed(window=4, ws=P, size=1 << 20, cu=P):
        return lib.fa_bwd_varlen_window(P, P, P, P, P, P, P, P, P, cu, 2, 10, 5, 2, 2, 64, 0.1,
                                        window, 0, ws, size, NULL)
    assert packed(window=0) == -1 and packed(cu=NULL) == -1 and packed(size=8) == -4


def test_workspace_sizes(lib):
    import exact_attention_33_gb300 as fa
    short = fa.fa_decode_window_workspace_size(4, 8, 2, 128, 100000, 64, 4)
    full = fa.fa_decode_workspace_size(4, 8, 2, 128, 100000)
    assert fa.FA_WORKSPACE_HEADER_BYTES < short < full
    # a window that covers the context needs what the plain call needs
    assert fa.fa_decode_window_workspace_size(4, 8, 2, 128, 1000, 5000, 0) == \
        fa.fa_decode_workspace_size(4, 8, 2, 128, 1000)
    assert fa.fa_bwd_window_workspace_size(1, 4, 2, 256, 64, 100) >= fa.fa_bwd_workspace_size(1, 4, 256)
    with pytest.raises(ValueError):
        fa.fa_bwd_window_workspace_size(1, 4, 2, 256, 64, 0)
    # the sinks' partial sums do not grow with sequences that are there already
    long, many = (fa.fa_bwd_window_workspace_size(n, 8, 8, 65536, 128, 64, 4) for n in (1, 1000))
    vectors = fa.fa_bwd_workspace_size(1000, 8, 65536)
    assert many - vectors < 8 * 1000 * 6 * 2 * 128 * 128 * 4
    assert long < 1 << 30


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    import exact_attention_33_gb300 as fa
    q = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for call in (lambda: fa.fa_fwd_window(q, q, q, 4),
                 lambda: fa.fa_bwd_window(q, q, q, q, torch.zeros(1, 2, 8), q, 4),
                 lambda: fa.fa_fwd_varlen_window(q[0], q[0], q[0], cu, 8, 4),
                 lambda: fa.fa_bwd_varlen_window(q[0], q[0], q[0], q[0], torch.zeros(2, 8), q[0],
                                                 cu, 8, 4),
                 lambda: fa.fa_decode_paged_window(q[0], q, q, cu[None], cu, 1, 4),
                 lambda: fa.fa_fwd_paged_window(q[0], q, q, cu[None], cu, cu, 8, 8, 4)):
        with pytest.raises(ValueError):
            call()


def rows(seed, *shape):
    torch = pytest.importorskip("torch")
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape))


def test_reference_without_a_window_is_the_oracle():
    import oracle
    import window_reference as ref
    q, k, v, g = (rows(i, 50, 16) for i in range(4))
    want, lse = oracle.attention_dense(*(x.numpy()[None, :, None] for x in (q, k, v)), causal=True)
    for window, sinks in ((50, 0), (1000, 3), (1, 50)):
        out, l, _ = ref.forward(q, k, v, window, sinks)
        assert np.abs(out.numpy() - want[0, :, 0]).max() < 1e-12
        assert np.abs(l.numpy() - lse[0, 0]).max() < 1e-12
        grads = ref.backward(q, k, v, g, window, sinks)[0]
        wants = oracle.attention_backward_dense(*(x.numpy()[None, :, None] for x in (q, k, v, g)),
                                                causal=True)
        for a, b in zip(grads, wants):
            assert np.abs(a.numpy() - b[0, :, 0]).max() < 1e-12


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (5, 0), (7, 3), (20, 25)])
def test_reference_by_hand_and_by_differences(window, sinks):
    """Each row recomputed over its visible keys alone; gradients against
    central differences."""
    import torch
    import window_reference as ref
    q, k, v, g = (rows(10 + i, 23, 4) for i in range(4))
    out, lse, _ = ref.forward(q, k, v, window, sinks)
    for p in range(23):
        js = [j for j in range(p + 1) if j > p - window or j < sinks]
        x = torch.stack([(q[p] * k[j]).sum() / 2.0 for j in js])
        assert torch.allclose(out[p], torch.softmax(x, 0) @ v[js], atol=1e-12)
        assert abs(float(lse[p] - torch.logsumexp(x, 0))) < 1e-12
    grads = ref.backward(q, k, v, g, window, sinks)[0]
    x = [q, k, v]
    for i in range(3):
        u = rows(20 + i, 23, 4)
        f = [float((ref.forward(*(t + h * u if j == i else t for j, t in enumerate(x)), window,
                                sinks)[0] * g).sum()) for h in (1e-5, -1e-5)]
        assert abs((f[0] - f[1]) / 2e-5 - float((grads[i] * u).sum())) < 1e-7
