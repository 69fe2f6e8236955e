"""Every value row of the 8-bit frame cache reaches the output with its own weight.

Over a long cache one wrong value row moves O by less than O's own rounding.  So V is zero here but for
one element a row, each in a column of its own: column c of O is then p_j v_j of a single key j, and a
row taken from another place, with another scale, dropped, or met by another key's weight
shows in full.  The keys are dealt over groups of d columns by a permutation until every key
has had its turn: the first and last of pages, of the kernels' steps, of ranges, and key n - 1.
"""
import math

import numpy as np
import pytest
import torch

from cache_helpers import random_pool, strided, tables
from gpu_helpers import sfa

pytestmark = pytest.mark.gpu

ROWS, TILES = 4, 8  # SFA_DEBUG_CACHE_*: the kernel of few rows, the kernel of many
U = 2.0 ** -8       # a bf16 rounding: of the probability, and of O


def _values(codes, scale):
    e = scale.view(torch.uint8).double() - 127
    return (codes.double().unflatten(-1, (-1, 32)) * torch.exp2(e).unsqueeze(-1)).flatten(-2)


CASES = [
    # B, Hk, G, L, d, page_len, kv, per_head, causal, ragged, flags
    (1, 2, 1, 1, 128, 64, 30000, True, False, False, 0),        # one token, ranges cut by the bound or dealt
    (2, 2, 1, 1, 64, 16, 9001, False, False, True, ROWS),
    (3, 2, 3, 1, 128, 40, 4099, True, False, True, ROWS),       # pages end inside a stretch
    (1, 3, 2, 5, 64, 7, 1500, True, True, True, ROWS),
    (2, 1, 1, 16, 128, 1560, 6000, False, True, True, ROWS),
    (1, 2, 2, 20, 64, 48, 2500, True, False, False, ROWS),      # two row tiles
    (1, 2, 1, 130, 128, 64, 4099, True, False, True, TILES),    # one token past a query tile
    (2, 2, 1, 100, 64, 16, 3000, False, False, True, TILES),    # one query tile
    (1, 3, 1, 300, 128, 40, 2111, True, True, True, TILES),
    (2, 2, 3, 111, 64, 7, 1800, True, True, True, TILES),
    (1, 4, 1, 260, 64, 200, 5000, True, False, True, TILES),
    (1, 12, 1, 513, 128, 1560, 3120, True, False, True, 0),     # several waves
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}H{}x{}L{}d{}P{}kv{}".format(*c[:7]) + {0: "", ROWS: "rows", TILES: "tiles"}[c[-1]])
def test_every_value_row_arrives(case):
    B, Hk, G, L, d, P, kv, per_head, causal, ragged, flags = case
    m, g = sfa(), np.random.default_rng(kv + L)
    heads, rows = (1, Hk) if per_head else (Hk, 1)
    N = -(-kv // P)
    n_pages = B * rows * N + 2
    cache = random_pool(g, m, n_pages, heads, P, d)
    table = torch.from_numpy(tables(g, B, rows, N, n_pages)).cuda()
    n = np.full((B, Hk), kv)
    if ragged:
        n = g.integers(kv // 3, kv + 1, (B, Hk))
        n[0, 0] = kv
    if not per_head:
        n[:] = n[:, :1]
    n = torch.from_numpy(n.astype(np.int32)).cuda()
    # pool places of every (b, key head, token); V: zeros at the smallest scale, NaN codes where nothing is
    j = torch.arange(kv, device="cuda")
    page = table.long()[..., j // P].expand(B, Hk, kv)
    head = (torch.arange(Hk, device="cuda") if heads > 1 else torch.zeros(Hk, dtype=torch.long, device="cuda"))[None, :, None].expand(B, Hk, kv)
    row = (j % P).expand(B, Hk, kv)
    there = j < n[..., None]
    codes, scale = cache.v.view(torch.uint8), cache.v_scale.view(torch.uint8)
    for t, s in ((codes, scale), (cache.k.view(torch.uint8), cache.k_scale.view(torch.uint8))):
        unused = torch.ones(t.shape[:3], dtype=torch.bool, device="cuda")
        unused[page[there], head[there], row[there]] = False
        t[unused] = 0x7f
        s[unused] = 0xfe
    k = torch.where(there[..., None], _values(cache.k, cache.k_scale)[page, head, row], 0.0)
    q = strided(torch.from_numpy(g.standard_normal((B, Hk * G, L, d))).bfloat16().cuda(), "blhd")
    x = torch.einsum("bhgid,bhjd->bhgij", q.double().reshape(B, Hk, G, L, d), k) / math.sqrt(d)
    seen = there[:, :, None, None, :]
    if causal:
        last = n.long()[:, :, None, None, None] - L + torch.arange(L, device="cuda")[:, None]
        seen = seen & (j <= last)
    p = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    reach = (q.double().abs().reshape(B, Hk, G, L, d) @ k.abs().transpose(-1, -2)[:, :, None]).amax().item() / math.sqrt(d)
    # a score is off by at most d + 4 roundings of 2^-24 of `reach`, and the sums by less than 2^-18
    slack = 2 * (d + 4) * 2.0 ** -24 * reach + 2.0 ** -18
    slot = torch.from_numpy(g.permutation(kv)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for group in range(-(-kv // d)):
        mine = (slot // d == group) & there
        v = torch.zeros(B, Hk, kv, d, dtype=torch.float64, device="cuda")
        codes[page[there], head[there], row[there]] = 0
        scale[page[there], head[there], row[there]] = 3
        b, h, at = mine.nonzero(as_tuple=True)
        col = slot[at] % d
        # four-bit numbers of either sign; every other group has exponents above 0 and above 7 too
        byte = torch.from_numpy(g.integers(0x38, 0x7f, len(at)) + 128 * g.integers(0, 2, len(at))).to(torch.uint8).cuda()
        e = torch.from_numpy(g.integers(-6, 10 if group % 2 else 1, len(at))).cuda()
        codes[page[b, h, at], head[b, h, at], row[b, h, at], col] = byte
        scale[page[b, h, at], head[b, h, at], row[b, h, at], col // 32] = (e + 127).to(torch.uint8)
        v[b, h, at, col] = byte.view(torch.float8_e4m3fn).double() * torch.exp2(e.double())
        want = (p @ v[:, :, None]).reshape(B, Hk * G, L, d)
        o, _ = m.forward_cache(q, cache, table, n if per_head else n[:, 0].contiguous(), causal=causal, max_kv=kv, H_kv=Hk,
                               dev_status=status, debug_flags=flags)
        bound = U * want.abs() + (U + slack) * (1 + U) * want.abs() + 1e-30
        off = (o.double() - want).abs() > bound
        assert not off.any(), (group, off.nonzero()[:4].tolist(), o[off][:4].tolist(), want[off][:4].tolist())
    torch.cuda.synchronize()
    assert status.item() == 0
