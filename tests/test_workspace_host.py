"""Workspace sizes (no GPU): a workspace sized for the largest batch and the
longest sequence serves every smaller one."""
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
