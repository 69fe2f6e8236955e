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
