"""How much workspace forward_cache asks for: the host's plan of key ranges (CPU)."""
import ctypes

import pytest

from test_cache_abi import GOOD, CacheAttnDesc, CacheDesc, sfa  # noqa: F401


def _workspace(sfa, B, H, Hk, Lq, d, kv, len_stride_h=0):  # noqa: F811
    desc = CacheAttnDesc(B, H, Hk, Lq, d, 0.125, 0, kv)
    for t in ("q", "o"):
        for i, s in enumerate((H * Lq * d, Lq * d, d)):
            setattr(desc, f"{t}_stride{i}", s)
    desc.len_stride_b, desc.len_stride_h = max(1, len_stride_h * Hk), len_stride_h
    cache = CacheDesc(4, Hk, 64, d, GOOD, GOOD, GOOD, GOOD, GOOD, -(-kv // 64), 0, 0)
    need = ctypes.c_size_t(0)
    assert sfa.load().sfa_forward_cache_workspace(ctypes.byref(desc), ctypes.byref(cache), ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("B,H,Hk,Lq,kv", [(1, 64, 8, 25600, 65536), (1, 12, 12, 63960, 32768), (4, 64, 8, 4096, 65536),
                                          (1, 12, 12, 16384, 8192), (1, 64, 8, 8192, 65536)])
def test_long_prefills_are_not_cut(sfa, B, H, Hk, Lq, kv):  # noqa: F811
    """Their partial results cost more than the ranges gain, and hundreds of MB of workspace."""
    assert _workspace(sfa, B, H, Hk, Lq, 128, kv) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", [1, 40, 700, 4680, 30000, 250000])
@pytest.mark.parametrize("kv", [1000, 100000, 1 << 29])
@pytest.mark.parametrize("heads", [0, 1])
def test_workspaces_are_bounded(sfa, d, Lq, kv, heads):  # noqa: F811
    for B, H, Hk in ((1, 1, 1), (1, 12, 12), (2, 64, 8), (16, 24, 24)):
        assert _workspace(sfa, B, H, Hk, Lq, d, kv, heads) <= 512 << 20


def test_few_rows_and_chunks_are_cut(sfa):  # noqa: F811
    """One token over long caches, and a streaming chunk, still run as several ranges."""
    rows = 12 * 4680
    assert _workspace(sfa, 1, 12, 12, 4680, 128, 20280, 1) == -(-3 * rows * 129 * 4 // 256) * 256
    assert _workspace(sfa, 8, 12, 12, 1, 128, 16384) >= 3 * 96 * 129 * 4
