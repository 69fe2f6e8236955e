"""The 8-bit frame cache's calls at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

from cache_helpers import random_pool
from gpu_helpers import sfa

pytestmark = pytest.mark.gpu


def _poison(*shapes):
    """NaN in freed blocks of the sizes that a call is about to allocate."""
    blocks = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("L", [5, 200])
def test_padded_rows_of_allocated_outputs(L):
    """They hold what a padded row stands for, not what the memory held before."""
    m, g = sfa(), np.random.default_rng(L)
    B, H, d = 2, 2, 64
    cache = random_pool(g, m, 10, H, 64, d)
    table = torch.arange(10, dtype=torch.int32, device="cuda").reshape(B, 5)
    lens = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    rows = torch.tensor([L // 2, 0], dtype=torch.int32, device="cuda")
    q, k, v = (torch.from_numpy(g.standard_normal((B, H, L, d))).bfloat16().cuda() for _ in range(3))
    bf, f32 = ((B, H, L, d), torch.bfloat16), ((B, H, L), torch.float32)
    _poison(bf, f32)
    o, l = m.forward_cache(q, cache, table, lens, q_lens=rows)
    _poison(bf)
    y = m.cache_append(m.cache_create(10, 64, d, heads=H), q, k, v, table, torch.zeros_like(lens), lens=rows)
    want_o, want_l = m.forward_cache(q, cache, table, lens)
    want_y, _ = m.qk_norm_rope(q)
    torch.cuda.synchronize()
    for b, n in enumerate(rows.tolist()):
        assert (o[b, :, n:] == 0).all() and torch.isneginf(l[b, :, n:]).all() and (y[b, :, n:] == 0).all()
        assert torch.equal(o[b, :, :n], want_o[b, :, :n]) and torch.equal(l[b, :, :n], want_l[b, :, :n])
        assert torch.equal(y[b, :, :n], want_y[b, :, :n])
    # outputs of the caller stay as they are there
    o2, l2, y2 = torch.full_like(q, 5.0), torch.full_like(l, 5.0), torch.full_like(q, 5.0)
    m.forward_cache(q, cache, table, lens, q_lens=rows, out=o2, lse=l2)
    m.cache_append(m.cache_create(10, 64, d, heads=H), q, k, v, table, torch.zeros_like(lens), lens=rows, q_out=y2)
    for b, n in enumerate(rows.tolist()):
        assert (o2[b, :, n:] == 5).all() and (l2[b, :, n:] == 5).all() and (y2[b, :, n:] == 5).all()


def test_nan_codes_and_scales_are_read_as_the_numbers_that_the_header_names():
    """Alone in a row, so that the attention of one key gives the row itself."""
    m, d = sfa(), 128
    rows = torch.zeros(6, d, dtype=torch.uint8)
    scale = torch.full((6, d // 32), 127, dtype=torch.uint8)
    rows[0, 5], rows[1, 70], rows[2, 127] = 0x7f, 0xff, 0x7f
    scale[2] = 200                     # 480 * 2^73
    rows[3, 9], scale[3] = 0x01, 255   # 2^-9 * 2^128
    rows[4, 9], scale[4] = 0x3c, 255   # 1.5 * 2^128: past bf16
    rows[5, 9], scale[5] = 0x38, 1     # 2^-126
    want = torch.zeros(6, d, dtype=torch.float64)
    want[0, 5], want[1, 70], want[2, 127] = 480.0, -480.0, 480.0 * 2.0 ** 73
    want[3, 9], want[4, 9], want[5, 9] = 2.0 ** 119, float("inf"), 2.0 ** -126
    cache = m.cache_create(6, 1, d)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8).copy_(rows.reshape(6, 1, 1, d))
        s.view(torch.uint8).copy_(scale.reshape(6, 1, 1, 4))
    table = torch.arange(6, dtype=torch.int32, device="cuda").reshape(6, 1)
    zero = torch.zeros(6, dtype=torch.int32, device="cuda")
    k, v = m.cache_read(cache, table, zero, 1)
    assert torch.equal(k[:, 0, 0].double().cpu(), want) and torch.equal(v[:, 0, 0].double().cpu(), want)
    finite = [0, 1, 2]  # (magnitudes of 2^100 and more may overflow in a partial result)
    for L, flags in ((1, m.SFA_DEBUG_CACHE_ROWS), (40, m.SFA_DEBUG_CACHE_TILES)):
        q = torch.zeros(6, 1, L, d, dtype=torch.bfloat16, device="cuda")
        o, l = m.forward_cache(q, cache, table, zero + 1, debug_flags=flags)
        torch.cuda.synchronize()
        assert torch.equal(o[finite].double().cpu(), want[finite][:, None, None].expand(3, 1, L, d))
        assert (l[finite] == 0).all()


@pytest.mark.parametrize("L,flags", [(1, 4), (20, 4), (100, 8), (300, 8)])
@pytest.mark.parametrize("kv", [100, 4000])
def test_attention_in_place(L, flags, kv):
    """O over its own queries: each is read before its row is written, keys in one range or several."""
    m, g = sfa(), np.random.default_rng(L)
    cache = random_pool(g, m, 20, 2, 200, 64)
    table = torch.arange(20, dtype=torch.int32, device="cuda").reshape(1, 20)
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(g.standard_normal((1, L, 6, 64))).bfloat16().cuda().transpose(1, 2)
    args = dict(causal=True, max_kv=kv, debug_flags=flags)
    o, l = m.forward_cache(q, cache, table, lens, **args)
    o2, l2 = m.forward_cache(q, cache, table, lens, out=q, **args)
    torch.cuda.synchronize()
    assert o2 is q and torch.equal(o2, o) and torch.equal(l2, l)
