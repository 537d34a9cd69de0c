"""Workspace sizes (no GPU): a workspace sized for the largest batch and the
longest sequence or context serves every smaller one."""
import itertools

import pytest


@pytest.fixture(scope="module")
def fa():
    from exact_attention_33_gb300.build import build
    build()
    import exact_attention_33_gb300 as fa_mod
    return fa_mod


def rises(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


LENGTHS = sorted({*range(1, 700, 37), *(128 * k + e for k in range(1, 40) for e in (-1, 0, 1)),
                  *(128 * k for k in range(40, 1100, 9)), 21120, 21248, 1 << 20})


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 300), (2, 128), (2, 129), (70, 16),
                                          (512, 16), (1000, 256), (4096, 4), (4096, 9000)])
def test_backward_size_rises_with_the_length(fa, window, sinks):
    for B, H, Hkv, d in ((16, 32, 8, 128), (1, 4, 4, 128), (1, 1, 1, 64), (700, 2, 2, 64)):
        assert rises([fa.fa_bwd_window_workspace_size(B, H, Hkv, n, d, window, sinks)
                      for n in LENGTHS]), (B, H, Hkv, d)


def test_backward_size_rises_with_the_batch(fa):
    for n, window, sinks in itertools.product((256, 1000, 21120), (1, 70, 512), (16, 200, 300)):
        assert rises([fa.fa_bwd_window_workspace_size(B, 8, 2, n, 128, window, sinks)
                      for B in range(1, 1200, 7)])


CONTEXTS = sorted({0, 1, *range(16, 2200, 60), 2048, 2049, *range(2200, 70000, 977), 1 << 20})


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 20), (2040, 4), (4096, 64)])
def test_decode_size_rises(fa, window, sinks):
    for H, Hkv, d in ((32, 8, 128), (8, 8, 64), (16, 1, 128)):
        size = [[fa.fa_decode_window_workspace_size(b, H, Hkv, d, n, window, sinks)
                 for n in CONTEXTS] for b in (1, 2, 3, 7, 8, 33, 64, 65, 200, 1000)]
        assert all(rises(row) for row in size) and all(rises(col) for col in zip(*size))
        if not window:
            assert size[6] == [fa.fa_decode_workspace_size(64, H, Hkv, d, n) for n in CONTEXTS]


def test_decode_size_stays_near_what_a_call_needs(fa):
    """Partial states of (o, m, l) for twice as many splits as work items that
    fill the GPU, or for splits of 512 keys, whichever is more."""
    for b, n in ((1, 100), (64, 2048), (64, 32768), (1, 1 << 20), (512, 4096)):
        got = fa.fa_decode_workspace_size(b, 32, 8, 128, n)
        rows = max(b * ((n + 511) // 512), min(b * ((n + 63) // 64), 2 * 14 * 160 // 8))
        assert got <= 256 + 32 * rows * (128 + 2) * 4 + 512, (b, n)
