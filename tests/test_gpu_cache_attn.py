"""Attention over the 8-bit frame cache against the float64 oracle on the cache's own values."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C

from cache_helpers import empty_pool, f64, gather, pool_values, random_pool, strided, tables
from gpu_helpers import sfa

pytestmark = pytest.mark.gpu

# O: the probabilities are rounded to bf16 (2^-8 of each, so 2^-8 of sum p|v|) and O once more
# (2^-8 of it).  fp32: a score is off by at most d + 4 roundings of 2^-24 of sum |q k| * scale
# plus the exponential's 2^-22, which moves a probability by that share; `slack` covers it and
# the fp32 sums.  LSE moves by the scores' error.
U = 2.0 ** -8


def check(o, lse, q, k, v, scale, causal, empty_ok=True):
    if q.shape[0] == 0:
        return
    want, wl, mag = C.attention(q, k, v, scale, causal)
    d = q.shape[-1]
    reach = scale * (np.abs(q) @ np.abs(k).T).max() if k.shape[0] else 0.0
    slack = 2 * (d + 4) * 2.0 ** -24 * reach + 2.0 ** -18
    o, lse = f64(o), f64(lse)
    bound = U * np.abs(want) + (U + slack) * (1 + U) * mag + 1e-30
    assert np.isfinite(o).all()
    err = np.abs(o - want)
    assert (err <= bound).all(), ((err - bound).max(), err.max())
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert (np.abs(lse[fin] - wl[fin]) <= slack + 2.0 ** -22 * np.abs(wl[fin])).all(), np.abs(lse[fin] - wl[fin]).max()


def poisoned(m, cache, table, lens, per_head):
    """Every row that no sequence uses gets NaN codes and the largest scale."""
    P, heads = cache.k.shape[2], cache.k.shape[1]
    used = np.zeros(tuple(cache.k.shape[:3]), bool)
    B, Hk = lens.shape
    for b in range(B):
        for h in range(Hk):
            for j in range(lens[b, h]):
                used[C.place(table, heads, P, b, h, j)] = True
    hide = torch.from_numpy(~used).cuda()
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8)[hide] = 0x7f
        s.view(torch.uint8)[hide] = 0xfe


def run_case(B, H, Hk, L, d, P, kv, per_head=False, causal=False, ragged=False, q_ragged=False, mem="bhld", seed=0,
             scale=None, max_kv=None, q_gain=1.0, flags=0, table_len=0):
    m, g = sfa(), np.random.default_rng(seed + 7 * L + kv + d)
    heads, rows = (1, Hk) if per_head else (Hk, 1)
    n = max(1, -(-kv // P))
    n_pages = B * rows * n + 2
    cache = random_pool(g, m, n_pages, heads, P, d)
    table = tables(g, B, rows, n, n_pages)
    lens = np.full((B, Hk), kv, np.int32)
    if ragged:
        lens = g.integers(0, kv + 1, (B, Hk)).astype(np.int32)
        lens[0, 0] = kv
        lens[-1, -1] = 0 if B * Hk > 1 else kv
    if not per_head:
        lens[:] = lens[:, :1]
    poisoned(m, cache, table, lens, per_head)
    if table_len > n:  # a table that could hold far more than it does
        table = np.concatenate([table, np.zeros((B, rows, table_len - n), np.int32)], 2)
    q_lens = None
    if q_ragged:
        q_lens = g.integers(0, L + 1, B).astype(np.int32)
    q = torch.from_numpy(q_gain * g.standard_normal((B, H, L, d))).bfloat16()
    qc = strided(q.cuda(), mem)
    if q_lens is not None:
        for b in range(B):
            qc[b, :, q_lens[b]:] = float("nan")
    out = strided(torch.full_like(q, 5.0).cuda(), mem)
    lse = torch.full((B, H, L), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(causal=causal, scale=scale, max_kv=(0 if table_len else kv) if max_kv is None else max_kv, H_kv=Hk, debug_flags=flags,
                q_lens=None if q_lens is None else torch.from_numpy(q_lens).cuda())
    t, ln = torch.from_numpy(table).cuda(), torch.from_numpy(lens if per_head else lens[:, 0].copy()).cuda()
    o, l = m.forward_cache(qc, cache, t, ln, out=out, lse=lse, dev_status=status, **args)
    torch.cuda.synchronize()
    assert status.item() == 0, m.error_string(status.item())
    assert o is out and l is lse
    sc = 1 / math.sqrt(d) if scale is None else scale
    for b in range(B):
        mq = L if q_lens is None else int(q_lens[b])
        assert (o[b, :, mq:] == 5).all() and (l[b, :, mq:] == 5).all()
        for h in range(H):
            hk = h // (H // Hk)
            k, v = gather(cache, table, b, hk, int(lens[b, hk]))
            check(o[b, h, :mq], l[b, h, :mq], f64(q[b, h, :mq]), k, v, sc, causal)
    return m, qc, cache, t, ln, o, l, args


SMALL = [
    dict(B=3, H=2, Hk=1, L=1, d=64, P=16, kv=100, q_ragged=True, seed=3),  # q_lens 0 and 1
    # one token
    dict(B=1, H=1, Hk=1, L=1, d=128, P=16, kv=1),
    dict(B=2, H=3, Hk=3, L=1, d=64, P=1, kv=5),
    dict(B=3, H=12, Hk=4, L=1, d=128, P=64, kv=333, ragged=True, per_head=True),
    dict(B=1, H=2, Hk=2, L=1, d=128, P=200, kv=4099, per_head=True),
    dict(B=2, H=24, Hk=1, L=1, d=64, P=40, kv=1000, ragged=True),
    # a few tokens
    dict(B=2, H=6, Hk=2, L=5, d=128, P=7, kv=77, causal=True, ragged=True),
    dict(B=1, H=4, Hk=4, L=16, d=64, P=16, kv=130, causal=True, mem="blhd"),
    dict(B=2, H=2, Hk=1, L=17, d=128, P=24, kv=63, q_ragged=True, mem="slice"),
    dict(B=2, H=3, Hk=3, L=9, d=64, P=16, kv=4, causal=True),   # rows that see nothing
    dict(B=2, H=2, Hk=2, L=4, d=128, P=16, kv=64, causal=True, ragged=True, q_ragged=True),
    dict(B=1, H=2, Hk=1, L=3, d=128, P=16, kv=0),
]


ROWS, TILES = 4, 8  # SFA_DEBUG_CACHE_*: the kernel of few rows, the kernel of many


@pytest.mark.parametrize("flags", [0, TILES])
@pytest.mark.parametrize("case", SMALL, ids=lambda c: "B{B}H{H}.{Hk}L{L}d{d}P{P}kv{kv}".format(**c))
def test_few_rows(case, flags):
    run_case(**case, flags=flags)


# Tables long enough that the few rows' ranges are cut by the lengths on the device
DEALT = [
    dict(B=3, H=4, Hk=2, L=1, d=128, P=64, kv=2000, ragged=True, per_head=True, table_len=1300),
    dict(B=2, H=9, Hk=3, L=6, d=64, P=40, kv=900, ragged=True, causal=True, q_ragged=True, table_len=2000),
    dict(B=5, H=5, Hk=5, L=1, d=64, P=16, kv=3000, ragged=True, table_len=6000),
    dict(B=2, H=2, Hk=2, L=17, d=128, P=7, kv=131, ragged=True, per_head=True, table_len=20000),
    dict(B=4, H=8, Hk=4, L=1, d=128, P=64, kv=1500, table_len=600),
    dict(B=2, H=4, Hk=2, L=2, d=128, P=64, kv=0, table_len=2000),
    dict(B=1, H=2, Hk=1, L=3, d=64, P=64, kv=50, table_len=8000),
]


@pytest.mark.parametrize("case", DEALT, ids=lambda c: "B{B}H{H}.{Hk}L{L}d{d}P{P}kv{kv}".format(**c))
def test_ranges_cut_by_the_lengths(case):
    m, q, cache, t, ln, o, l, args = run_case(**case)
    # a captured call cuts them by the lengths that it finds
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(o), torch.zeros_like(l)
    ws = torch.empty(m.forward_cache_workspace_bytes(q, cache, t, ln, max_kv=args["max_kv"], H_kv=args["H_kv"]),
                     dtype=torch.uint8, device="cuda")
    kept = ln.clone()
    ln.zero_()
    with torch.cuda.graph(graph):
        m.forward_cache(q, cache, t, ln, out=out, lse=lse, workspace=ws, **args)
    graph.replay()
    ln.copy_(kept)
    graph.replay()
    torch.cuda.synchronize()
    for b in range(case["B"]):
        n = case["L"] if args["q_lens"] is None else int(args["q_lens"][b])
        assert torch.equal(out[b, :, :n], o[b, :, :n]) and torch.equal(lse[b, :, :n], l[b, :, :n])


CHUNKS = [
    dict(B=1, H=2, Hk=2, L=129, d=128, P=200, kv=600, per_head=True),
    dict(B=1, H=1, Hk=1, L=128, d=64, P=128, kv=128),
    dict(B=2, H=4, Hk=2, L=150, d=64, P=16, kv=413, causal=True, ragged=True),
    dict(B=1, H=3, Hk=1, L=300, d=128, P=40, kv=300, causal=True),
    dict(B=2, H=2, Hk=2, L=200, d=128, P=24, kv=100, causal=True, q_ragged=True, mem="slice"),
    dict(B=1, H=6, Hk=3, L=333, d=64, P=1560, kv=1560, per_head=True, mem="blhd"),
    dict(B=3, H=2, Hk=2, L=70, d=128, P=64, kv=900, ragged=True, per_head=True, q_ragged=True),
    dict(B=1, H=2, Hk=2, L=513, d=128, P=64, kv=257),
    dict(B=1, H=8, Hk=2, L=64, d=64, P=100, kv=2111, per_head=True),
    dict(B=1, H=1, Hk=1, L=260, d=128, P=16, kv=0),
]


@pytest.mark.parametrize("flags", [0, ROWS, TILES])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "B{B}H{H}.{Hk}L{L}d{d}P{P}kv{kv}".format(**c))
def test_chunks(case, flags):
    run_case(**case, flags=flags)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L", [1, 140])
def test_repeated_calls_and_the_bound_of_lengths(L, flags):
    """The result does not depend on what the workspace held, and max_kv is a matter of speed."""
    m, q, cache, t, ln, o, l, args = run_case(B=2, H=2, Hk=2, L=L, d=128, P=32, kv=1500, ragged=True, flags=flags)
    args.pop("max_kv")
    for max_kv in (0, 100, 1500, 48000):
        need = 64 * 4 * q.numel() // 128 * 129  # as much as 64 ranges take
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        o1, l1 = m.forward_cache(q, cache, t, ln, workspace=ws, max_kv=max_kv, **args)
        o2, l2 = m.forward_cache(q, cache, t, ln, max_kv=max_kv, **args)
        torch.cuda.synchronize()
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
        assert torch.allclose(o1.float(), o.float(), atol=2e-2, rtol=2 * U) and torch.allclose(l1, l, atol=1e-4)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L", [3, 200])
@pytest.mark.parametrize("gain", [30.0, 1e-3])
def test_sharp_and_flat_scores(L, gain, flags):
    # growing maxima (a late key that beats the earlier ones by far) and equal scores
    run_case(B=1, H=2, Hk=1, L=L, d=128, P=64, kv=700, q_gain=gain, flags=flags)
    run_case(B=1, H=2, Hk=1, L=L, d=64, P=64, kv=700, q_gain=gain, causal=True, flags=flags)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L", [3, 100, 200])
def test_scores_that_grow_from_key_to_key(L, flags):
    """Every key beats the ones before by more than the running maximum may lag: each chunk of
    every tile rescales what came before."""
    m, d, n = sfa(), 64, 300
    cache = empty_pool(m, 19, 1, 16, d)
    k = torch.zeros(1, 1, n, d)
    k[..., 0] = torch.arange(n).float() * 0.5  # scores 0.125 * 64 * 0.5 j = 4 j: a factor e^4 from key to key
    v = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1))
    table = torch.arange(19, dtype=torch.int32, device="cuda").reshape(1, 19)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, k.bfloat16().cuda(), v.bfloat16().cuda(), table, zero)
    q = torch.zeros(1, 1, L, d)
    q[..., 0] = 64.0
    q[..., 1:] = torch.randn(L, d - 1, generator=torch.Generator().manual_seed(2))
    q = q.bfloat16().cuda()
    kk, vv = gather(cache, table.unsqueeze(1).cpu().numpy(), 0, 0, n)
    for causal in (False, True):
        o, l = m.forward_cache(q, cache, table, zero + n, causal=causal, debug_flags=flags)
        torch.cuda.synchronize()
        check(o[0, 0], l[0, 0], f64(q[0, 0]), kk, vv, 0.125, causal)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L", [2, 150])
def test_large_scales_take_the_second_product(L, flags):
    """Blocks with exponents above 7 (magnitudes of 57344 and more), next to ordinary ones."""
    m, g = sfa(), np.random.default_rng(3)
    d, n = 128, 200
    cache = random_pool(g, m, 4, 1, 64, d)
    for s, to in ((cache.k_scale, 140), (cache.v_scale, 200)):
        b = s.view(torch.uint8)
        b[1:3, :, ::3, 1] = to
    table = np.array([[[2, 0, 1, 3]]], np.int32)
    q = torch.from_numpy(1e-5 * g.standard_normal((1, 1, L, d))).bfloat16()
    o, l = m.forward_cache(q.cuda(), cache, torch.from_numpy(table).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                           debug_flags=flags)
    torch.cuda.synchronize()
    k, v = gather(cache, table, 0, 0, n)
    check(o[0, 0], l[0, 0], f64(q[0, 0]), k, v, 1 / math.sqrt(d), False)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L", [1, 130])
@pytest.mark.parametrize("what", ["length", "negative length", "page"])
def test_bad_lengths_and_pages_are_reported(L, what, flags):
    m, g = sfa(), np.random.default_rng(4)
    cache = random_pool(g, m, 6, 1, 16, 64)
    table = np.array([[[0, 1, 2]], [[3, 4, 5]]], np.int32)
    lens = np.array([40, 48], np.int32)
    q = torch.from_numpy(g.standard_normal((2, 1, L, 64))).bfloat16().cuda()
    if what == "length":
        lens[1] = 49
    elif what == "negative length":
        lens[1] = -1
    else:
        table[1, 0, 1] = 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = m.forward_cache(q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), dev_status=status,
                           debug_flags=flags)
    torch.cuda.synchronize()
    assert status.item() == m.SFA_ERR_BAD_SET
    k, v = gather(cache, table, 0, 0, 40)  # the other sequence is right
    check(o[0, 0], l[0, 0], f64(q[0, 0]), k, v, 0.125, False)


@pytest.mark.parametrize("L", [1, 129])
def test_other_stream_and_graph_replay(L):
    m, q, cache, t, ln, o, l, args = run_case(B=1, H=2, Hk=2, L=L, d=64, P=32, kv=900, flags=TILES if L > 1 else ROWS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o1, l1 = m.forward_cache(q, cache, t, ln, **args)
    side.synchronize()
    assert torch.equal(o1, o) and torch.equal(l1, l)
    o2, l2 = torch.zeros_like(q), torch.zeros_like(l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward_cache(q, cache, t, ln, out=o2, lse=l2, **args)
    ln.fill_(333)  # a replay reads the lengths and tables as they are then
    want = m.forward_cache(q, cache, t, ln, **args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, want[0]) and torch.equal(l2, want[1])


@pytest.mark.parametrize("Lq", [1, 24, 200])
def test_a_streaming_layer(Lq):
    """Chunk after chunk as a streaming layer runs them: norm and rotation, the append, the
    attention over the heads' own caches, merged by LSE with a branch over other frames."""
    m, g = sfa(), np.random.default_rng(11)
    B, H, d, P = 1, 4, 128, 24
    Hk, n_pages = H, 4 * 40
    cache = empty_pool(m, n_pages, 1, P, d)
    table = torch.from_numpy(tables(g, B, Hk, 30, n_pages)).cuda()
    lens = torch.zeros(B, Hk, dtype=torch.int32, device="cuda")
    rope = m.rope_table((44, 42, 42))
    w = torch.from_numpy(1 + 0.1 * g.standard_normal((2, d))).float().cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(3):
        q, k, v = (torch.from_numpy(g.standard_normal((B, H, Lq, d))).bfloat16().cuda() for _ in range(3))
        pos = torch.from_numpy(g.integers(0, 50, (B, Lq, 3)).astype(np.int32)).cuda()
        args = dict(rope=rope, positions=pos, q_weight=w[0], k_weight=w[1])
        qr = m.cache_append(cache, q, k, v, table, lens, dev_status=status, **args)
        lens = lens + Lq
        o, l = m.forward_cache(qr, cache, table, lens, causal=True, max_kv=3 * Lq, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        n = (step + 1) * Lq
        for h in range(H):
            kk, vv = gather(cache, table.cpu().numpy(), 0, h, n)
            check(o[0, h], l[0, h], f64(qr[0, h]), kk, vv, 1 / math.sqrt(d), True)
    # the whole cache = its first tokens merged with the others (tables split at a page)
    whole = m.forward_cache(qr, cache, table, lens)
    cut = min(3 * Lq // P, 1) * P
    if cut:
        first = m.forward_cache(qr, cache, table, torch.full_like(lens, cut))
        rest = m.forward_cache(qr, cache, table[:, :, 1:], lens - cut)
        both = m.lse_merge(first[0], first[1], rest[0], rest[1])
        torch.cuda.synchronize()
        assert torch.allclose(both[1], whole[1], atol=1e-5)
        assert torch.allclose(both[0].float(), whole[0].float(), atol=4 * U * 4)
    # the cache read back is what the bf16 attention over the same keys sees
    ko, vo = m.cache_read(cache, table, torch.zeros(B, dtype=torch.int32, device="cuda"), int(lens[0, 0]))
    L = int(lens[0, 0])
    ones = torch.ones(H, 1, dtype=torch.int32, device="cuda")
    dense = m.forward(qr[:, :, :Lq], ko[:, :, :Lq].contiguous(), vo[:, :, :Lq].contiguous(),
                      torch.zeros(H, 1, 1, dtype=torch.int32, device="cuda"), ones, Lq)
    part = m.forward_cache(qr, cache, table, torch.full_like(lens, Lq))
    torch.cuda.synchronize()
    assert L == 3 * Lq and torch.allclose(dense[1], part[1], atol=1e-4)
    assert torch.allclose(dense[0].float(), part[0].float(), atol=4 * U * 4)


def test_offsets_past_32_bits():
    """The last page of a pool of more than 2^32 bytes."""
    m, g = sfa(), np.random.default_rng(12)
    P, d = 4096, 128
    n_pages = (1 << 32) // (P * d) + 4
    cache = m.cache_create(n_pages, P, d)
    x = torch.randn(1, 1, 300, d, device="cuda").bfloat16()
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, x, x, table, zero)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    back = C.dequantise(*C.quantise(f64(x[0, 0])))
    for L, flags in ((1, ROWS), (150, TILES)):
        q = torch.randn(1, 1, L, d, device="cuda").bfloat16()
        o, l = m.forward_cache(q, cache, table, n, debug_flags=flags)
        torch.cuda.synchronize()
        check(o[0, 0], l[0, 0], f64(q[0, 0]), back, back, 1 / math.sqrt(d), False)


def test_a_wait_that_runs_out_is_reported():
    """The softmax withholds its first probabilities (a test hook): the waits run out after their
    limit, the call reports it and returns, and the next call is right."""
    m, q, cache, t, ln, o, l, args = run_case(B=1, H=2, Hk=2, L=300, d=128, P=32, kv=700, flags=TILES)
    for n in (300, 100):  # two query tiles, one
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        args["debug_flags"] = TILES | m.SFA_DEBUG_STALL_SOFTMAX
        m.forward_cache(q[:, :, :n], cache, t, ln, dev_status=status, timeout_us=2000, **args)
        torch.cuda.synchronize()
        assert status.item() == m.SFA_ERR_TIMEOUT
        status.zero_()
        args["debug_flags"] = TILES
        o2, l2 = m.forward_cache(q, cache, t, ln, dev_status=status, **args)
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.equal(o2, o) and torch.equal(l2, l)


def test_the_choice_of_kernel_by_size():
    """Rows and work on both sides of the choice, without a hook."""
    for L, B in ((31, 1), (32, 2), (33, 1), (40, 5)):
        run_case(B=B, H=4, Hk=4, L=L, d=64, P=32, kv=1100, ragged=True)
    run_case(B=2, H=6, Hk=6, L=130, d=128, P=64, kv=1400, per_head=True, causal=True)


def test_what_a_call_allocates_follows_its_stream():
    """Neither the zero fill of cache_read's outputs nor a reuse of forward_cache's workspace may
    be ordered by another stream than the call's."""
    m, g = sfa(), np.random.default_rng(5)
    cache = random_pool(g, m, 40, 2, 64, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(1, 40)
    lens = torch.tensor([2500], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(g.standard_normal((1, 2, 1, 64))).bfloat16().cuda()
    k0, v0 = m.cache_read(cache, table, start, 300)
    o0, l0 = m.forward_cache(q, cache, table, lens)
    need = m.forward_cache_workspace_bytes(q, cache, table, lens)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)  # the current stream is behind
        k1, v1 = m.cache_read(cache, table, start, 300, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(k1, k0) and torch.equal(v1, v0)
        with torch.cuda.stream(side):  # and now the other one
            torch.cuda._sleep(20_000_000)
        o1, l1 = m.forward_cache(q, cache, table, lens, stream=stream)
        others = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in (need, need, need)]
        torch.cuda.synchronize()
        assert torch.equal(o1, o0) and torch.equal(l1, l0) and all((x == 0xff).all() for x in others)


@pytest.mark.parametrize("flags", [ROWS, TILES])
@pytest.mark.parametrize("L,kv", [(3, 90), (3, 6000), (150, 700)])
def test_a_query_with_nan_answers_nan(L, kv, flags):
    """In its own row and no other, with the keys in one range and in several."""
    m, g = sfa(), np.random.default_rng(kv)
    cache = random_pool(g, m, 100, 1, 64, 64)
    table = g.permutation(100).astype(np.int32).reshape(1, 1, 100)
    q = torch.from_numpy(g.standard_normal((1, 1, L, 64))).bfloat16()
    q[0, 0, 1, 5] = float("nan")
    o, l = m.forward_cache(q.cuda(), cache, torch.from_numpy(table).cuda(),
                           torch.tensor([kv], dtype=torch.int32, device="cuda"), debug_flags=flags)
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 1]).all() and torch.isnan(l[0, 0, 1])
    rest = [i for i in range(L) if i != 1]
    k, v = gather(cache, table, 0, 0, kv)
    check(o[0, 0, rest], l[0, 0, rest], f64(q[0, 0, rest]), k, v, 0.125, False)


def test_calls_of_two_threads():
    """Each thread has a stream and outputs of its own; the cache is read by both."""
    from concurrent.futures import ThreadPoolExecutor
    m, g = sfa(), np.random.default_rng(11)
    cache = random_pool(g, m, 40, 2, 64, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(1, 40)
    lens = torch.tensor([2500], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    qs = [torch.from_numpy(g.standard_normal((1, 4, n, 64))).bfloat16().cuda() for n in (1, 200)]
    want = [(m.forward_cache(q, cache, table, lens), m.cache_read(cache, table, start, 300)) for q in qs]
    torch.cuda.synchronize()

    def work(q):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            r = [(m.forward_cache(q, cache, table, lens), m.cache_read(cache, table, start, 300)) for _ in range(50)]
        stream.synchronize()
        return r
    with ThreadPoolExecutor(2) as ex:
        for w, got in zip(want, ex.map(work, qs)):
            for r in got:
                for a, b in zip(w, r):
                    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


DEALT = [  # B, Hk, G, L, d, kv, page_len, causal, flags, max_kv as a share of kv
    (2, 8, 1, 1, 64, 30000, 64, False, ROWS, 1.0),
    (2, 8, 2, 5, 128, 30000, 40, True, ROWS, 1.0),
    (37, 3, 1, 1, 64, 4300, 16, False, ROWS, 1.0),
    (3, 11, 1, 100, 64, 2000, 16, True, TILES, 1.0),
    (3, 11, 1, 70, 128, 1500, 40, False, TILES, 0.3),
    (2, 2, 3, 290, 128, 3000, 64, True, TILES, 1.0),
    (1, 5, 1, 600, 64, 2500, 200, True, TILES, 1.5),
    (64, 1, 1, 130, 64, 700, 16, False, TILES, 1.0),
]


@pytest.mark.parametrize("how", ["one", "spread", "nothing", "all but one", "twos"])
@pytest.mark.parametrize("case", DEALT)
def test_uneven_caches_share_the_gpu(case, how):
    """Ranges dealt out by the lengths on the device: a long cache among short ones, empty ones,
    bounds that are too small, more caches than a warp has lanes, several row tiles."""
    B, Hk, G, L, d, kv, P, causal, flags, share = case
    m, g = sfa(), np.random.default_rng(kv + L)
    cache = random_pool(g, m, 50, 1, P, d)
    table = g.integers(0, 50, (B, Hk, -(-kv // P))).astype(np.int32)
    n = {"one": np.full((B, Hk), kv // 9), "spread": g.integers(0, kv + 1, (B, Hk)), "nothing": np.zeros((B, Hk)),
         "all but one": np.full((B, Hk), kv), "twos": kv // (1 + np.arange(B * Hk).reshape(B, Hk) % 2)}[how].astype(np.int32)
    n[-1, -1] = {"one": kv, "all but one": 1}.get(how, n[-1, -1])
    q = torch.from_numpy(g.standard_normal((B, Hk * G, L, d))).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = m.forward_cache(q.cuda(), cache, torch.from_numpy(table).cuda(), torch.from_numpy(n).cuda(), causal=causal,
                           max_kv=max(1, int(share * kv)), dev_status=status, debug_flags=flags)
    torch.cuda.synchronize()
    assert status.item() == 0
    empty = torch.from_numpy(np.repeat(n == 0, G, 1))
    assert (o.cpu()[empty] == 0).all() and torch.isneginf(l.cpu()[empty]).all() and torch.isfinite(o).all()
    (kc, ke), (vc, ve) = pool_values(cache)
    k_all, v_all = C.dequantise(kc, ke)[:, 0], C.dequantise(vc, ve)[:, 0]
    caches = [(b, h) for b in range(B) for h in range(Hk)]
    some = caches if kv * L < 100000 else caches[:3] + caches[-3:]
    for b, h in some[:40] + some[-1:]:
        at = table[b, h].astype(int)
        k, v = (x[at].reshape(-1, d)[: n[b, h]] for x in (k_all, v_all))
        for i in range(G):
            check(o[b, h * G + i], l[b, h * G + i], f64(q[b, h * G + i]), k, v, 1 / math.sqrt(d), causal)


@pytest.mark.parametrize("B,Hk,L", [(1, 12, 40), (2, 3, 300), (1, 16, 1)])
@pytest.mark.parametrize("shape", ["heads", "shared", "one"])
def test_workspace_bytes_are_those_of_the_call(B, Hk, L, shape):
    m, g = sfa(), np.random.default_rng(L)
    cache = random_pool(g, m, 40, 1, 64, 64)
    table = torch.from_numpy(g.integers(0, 40, (B, Hk, 600)).astype(np.int32)).cuda()
    n = torch.from_numpy(g.integers(2000, 600 * 64, (B, Hk)).astype(np.int32)).cuda()
    n = {"heads": n, "shared": n[:, :1].contiguous(), "one": n[:, 0].contiguous()}[shape]
    q = torch.from_numpy(g.standard_normal((B, Hk, L, 64))).bfloat16().cuda()
    size = m.forward_cache_workspace_bytes(q, cache, table, n)
    ws = torch.full((size + 256,), 0xff, dtype=torch.uint8, device="cuda")
    o1, l1 = m.forward_cache(q, cache, table, n, workspace=ws[:size])
    o2, l2 = m.forward_cache(q, cache, table, n)
    torch.cuda.synchronize()
    assert size > 0 and torch.equal(o1, o2) and torch.equal(l1, l2) and (ws[size:] == 0xff).all()
