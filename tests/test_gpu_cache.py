"""Norm and rotation, writing and reading of the 8-bit frame cache against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import cache as C

from cache_helpers import empty_pool, f64, pool_values, random_pool, strided, tables
from gpu_helpers import sfa

pytestmark = pytest.mark.gpu

# bf16 rounding is off by at most 2^-8 of the value; the fp32 work before it (a norm with a
# sum of at most 128 squares, reciprocal square root, sine, cosine and four products) stays
# below 16 roundings of 2^-24, i.e. 2^-20, of the magnitudes that are added
U_BF16, FP32 = 2.0 ** -8, 2.0 ** -20
TINY = 2.0 ** -133


def _close(got, want, mag):
    err = np.abs(f64(got) - want)
    bound = U_BF16 * np.abs(want) + (1 + U_BF16) * FP32 * mag + TINY
    assert (err <= bound).all(), (err - bound).max()


def _rope(m, axes, far):
    rope = m.rope_table(axes, scaling="yarn" if far else "none", factor=8.0 if far else 1.0, original_len=4096)
    return rope, rope.inv_freq.cpu().numpy()


def _positions(g, B, L, n, far):
    lo, hi = (-(1 << 21), 1 << 30) if far else (0, 2000)
    return torch.from_numpy(g.integers(lo, hi, (B, L, n)).astype(np.int32))


NORM_CASES = [
    # B, H, Hk, L, d, axes, layout, eps, weights, far, layout in memory
    (1, 1, 1, 1, 128, (128,), "half", 1e-6, True, False, "bhld"),
    (2, 12, 12, 1, 128, (64,), "half", 1e-6, True, True, "bhld"),
    (3, 6, 2, 37, 128, (44, 42, 42), "interleaved", 1e-6, True, False, "blhd"),
    (1, 5, 3, 1561, 64, (22, 10), "interleaved", 1e-5, False, True, "slice"),
    (2, 3, 1, 130, 64, (16, 24, 24), "half", None, True, False, "blhd"),
    (1, 16, 8, 9, 64, (0, 48), "half", 1e-6, False, False, "slice"),
    (1, 2, 2, 4099, 128, (2, 0, 4, 8), "interleaved", None, False, True, "bhld"),
    (4, 7, 7, 11, 128, None, "interleaved", 1e-6, True, False, "bhld"),
    # several tokens a warp
    (1, 2, 1, 9001, 128, (64,), "half", 1e-6, True, True, "blhd"),
    (3, 1, 1, 1999, 64, (22, 10), "interleaved", 1e-6, True, False, "slice"),
    (2, 4, 4, 2600, 128, None, "interleaved", 1e-6, True, False, "bhld"),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"B{c[0]}H{c[1]}.{c[2]}L{c[3]}d{c[4]}{c[6]}")
def test_norm_rope(case):
    B, H, Hk, L, d, axes, layout, eps, weights, far, mem = case
    m, g = sfa(), np.random.default_rng(L + d + H)
    q = strided(torch.from_numpy(g.standard_normal((B, H, L, d))).bfloat16().cuda(), mem)
    k = strided(torch.from_numpy(3 * g.standard_normal((B, Hk, L, d))).bfloat16().cuda(), mem)
    qw, kw = (torch.from_numpy(1 + 0.2 * g.standard_normal(d)).float() if weights else None for _ in range(2))
    rope = pos = None
    kw_o = dict()
    if axes:
        rope, f = _rope(m, axes, far)
        pos = _positions(g, B, L, len(axes), far)
        kw_o = dict(positions=pos.numpy(), inv_freq=f, axis_pairs=rope.axis_pairs, scale=rope.scale, layout=layout)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = dict(rope=rope, positions=cuda(pos), q_weight=cuda(qw), k_weight=cuda(kw), eps=eps, layout=layout)
    yq, yk = m.qk_norm_rope(q, k, **args)
    torch.cuda.synchronize()
    for x, y, w in ((q, yq, qw), (k, yk, kw)):
        want, mag = C.norm_rope(f64(x), None if w is None else w.numpy(), eps, **kw_o)
        _close(y, want, mag)
    # one of the two alone, and in place
    only, none = m.qk_norm_rope(q, **args)
    assert none is None and torch.equal(only, yq)
    _, only = m.qk_norm_rope(None, k, **args)
    assert torch.equal(only, yk)
    q2, k2 = q.clone(), k.clone()
    m.qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **args)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)


def test_norm_rope_zero_rows_and_shared_positions():
    m = sfa()
    q = torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16, device="cuda")
    q[1] = 1.0
    pos = torch.arange(5, dtype=torch.int32, device="cuda").unsqueeze(-1)
    rope = m.rope_table((64,))
    y, _ = m.qk_norm_rope(q, rope=rope, positions=pos)
    y2, _ = m.qk_norm_rope(q, rope=rope, positions=pos.expand(2, 5, 1).contiguous())
    assert (y[0] == 0).all() and torch.equal(y, y2)  # mean 0: eps keeps the norm finite
    # rows are independent: a non-finite one leaves the others alone, unrotated elements too
    q[0, 1, 2] = float("inf")
    y3, _ = m.qk_norm_rope(q, rope=m.rope_table((32,)), positions=pos)
    keep = torch.ones(2, 3, 5, dtype=torch.bool, device="cuda")
    keep[0, 1, 2] = False
    assert torch.isfinite(y3[keep].float()).all() and torch.isnan(y3[0, 1, 2].float()).all()
    q[0, 1, 2] = 1.0
    q[0, 1, 2, 40] = float("inf")
    y4, _ = m.qk_norm_rope(q, rope=m.rope_table((32,)), positions=pos, eps=None)
    assert torch.isfinite(y4[0, 1, 2, :40].float()).all() and y4[0, 1, 2, 40] == float("inf")


def test_long_context_tables():
    m = sfa()
    base = m.rope_table((64,)).inv_freq
    lin = m.rope_table((64,), scaling="linear", factor=4.0)
    assert torch.allclose(lin.inv_freq * 4, base, rtol=1e-15) and lin.scale == 1.0
    ntk = m.rope_table((64,), scaling="ntk", factor=4.0).inv_freq
    # ntk: the fastest pair is kept, the slowest slowed by the factor
    assert ntk[0] == base[0] and abs((base[-1] / ntk[-1]).item() - 4.0) < 1e-12
    yarn = m.rope_table((64,), scaling="yarn", factor=4.0, original_len=2048)
    ratio = base / yarn.inv_freq
    assert ratio[0] == 1.0 and abs(ratio[-1].item() - 4.0) < 1e-12 and (ratio[1:] >= ratio[:-1]).all()
    assert abs(yarn.scale - (0.1 * np.log(4.0) + 1)) < 1e-15


WRITE_CASES = [
    # B, Hk, L, d, page_len, per_head, ragged, memory
    (1, 1, 1, 128, 1, False, False, "bhld"),
    (2, 3, 1, 64, 16, False, False, "bhld"),
    (3, 5, 37, 128, 7, True, True, "blhd"),
    (2, 4, 333, 64, 40, False, True, "slice"),
    (1, 12, 200, 128, 1560, True, False, "blhd"),
]


def _write_setup(case, seed=0):
    B, Hk, L, d, P, per_head, ragged, mem = case
    m, g = sfa(), np.random.default_rng(seed + L + d)
    heads, rows = (1, Hk) if per_head else (Hk, 1)
    n = -(-(L + 2 * P) // P)
    n_pages = B * rows * n + 3
    table = tables(g, B, rows, n, n_pages)
    start = g.integers(0, 2 * P, (B, Hk) if per_head else (B,)).astype(np.int32)
    lens = g.integers(0, L + 1, B).astype(np.int32) if ragged else None
    k = torch.from_numpy(g.standard_normal((B, Hk, L, d)) * np.exp(2 * g.standard_normal((B, Hk, L, 1)))).bfloat16()
    v = torch.from_numpy(g.standard_normal((B, Hk, L, d))).bfloat16()
    cache = empty_pool(m, n_pages, heads, P, d)
    return m, cache, strided(k.cuda(), mem), strided(v.cuda(), mem), table, start, lens


def _expected_pool(cache, k, v, table, start, lens):
    pools = pool_values(cache)
    P, heads = cache.k.shape[2], cache.k.shape[1]
    B, Hk, L, _ = k.shape
    for (codes, e), x in zip(pools, (f64(k), f64(v))):
        c_new, e_new = C.quantise(x)
        for b in range(B):
            for h in range(Hk):
                s = int(start[b, h] if start.ndim == 2 else start[b])
                for i in range(L if lens is None else int(lens[b])):
                    at = C.place(table, heads, P, b, h, s + i)
                    codes[at], e[at] = c_new[b, h, i], e_new[b, h, i]
    return pools


def _gpu(x):
    return None if x is None else torch.from_numpy(x).cuda()


@pytest.mark.parametrize("case", WRITE_CASES, ids=lambda c: f"B{c[0]}H{c[1]}L{c[2]}d{c[3]}P{c[4]}")
def test_write_and_read_back(case):
    m, cache, k, v, table, start, lens = _write_setup(case)
    want = _expected_pool(cache, k, v, table, start, lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, k, v, _gpu(table), _gpu(start), lens=_gpu(lens), dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for (codes, e), (wc, we) in zip(pool_values(cache), want):  # untouched rows too
        np.testing.assert_array_equal(codes, wc)
        np.testing.assert_array_equal(e, we)
    L = case[2]
    ko, vo = m.cache_read(cache, _gpu(table), _gpu(start), L, lens=_gpu(lens), H_kv=k.shape[1], dev_status=status)
    ko2 = torch.full_like(k, 5.0)
    vo2 = torch.full_like(v, 5.0)
    m.cache_read(cache, _gpu(table), _gpu(start), L, lens=_gpu(lens), k_out=ko2, v_out=vo2)
    torch.cuda.synchronize()
    assert status.item() == 0
    for got, got2, x in ((ko, ko2, k), (vo, vo2, v)):
        back = C.dequantise(*C.quantise(f64(x)))
        for b in range(k.shape[0]):
            n = L if lens is None else int(lens[b])
            np.testing.assert_array_equal(f64(got[b, :, :n]), back[b, :, :n])
            np.testing.assert_array_equal(f64(got2[b, :, :n]), back[b, :, :n])
            assert (got[b, :, n:] == 0).all() and (got2[b, :, n:] == 5).all()


def test_every_code_and_scale_reads_back_exactly():
    m = sfa()
    codes = torch.arange(256, dtype=torch.uint8)
    codes[[0x7f, 0xff]] = 0  # NaN codes are never written
    n = 244  # scale bytes 3 .. 246
    rows = codes.reshape(2, 128)
    cache = m.cache_create(1, 2 * n, 128)
    k = rows.repeat(n, 1)
    e = torch.arange(3, 3 + n, dtype=torch.uint8).repeat_interleave(2).unsqueeze(1).expand(2 * n, 4)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8).copy_(k.reshape(1, 1, 2 * n, 128))
        s.view(torch.uint8).copy_(e.reshape(1, 1, 2 * n, 4))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ko, vo = m.cache_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), 2 * n)
    want = C.dequantise(k.view(torch.float8_e4m3fn).double().numpy(), e.numpy().astype(np.int64) - 127)
    np.testing.assert_array_equal(f64(ko[0, 0]), want)
    np.testing.assert_array_equal(f64(vo[0, 0]), want)


def test_block_values_at_the_edges():
    """Blocks of zeros, of the smallest and largest bf16 numbers, of midpoints, of one large
    value among small ones."""
    m = sfa()
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros(8, 128)
    x[1] = 2.0 ** -133
    x[2] = big
    x[3, ::2], x[3, 1::2] = big, 2.0 ** -133
    x[4] = torch.linspace(-448, 448, 128)
    x[5, :32], x[5, 32:64], x[5, 64:96], x[5, 96:] = 448.0, 450.0, 224.0, -226.0
    x[6] = torch.tensor([17.0, 18.0, 19.0, 21.0, 23.0, 25.0, 27.0, 29.0]).repeat(16)  # halfway between codes
    x[7, 5] = 1e30
    x = x.bfloat16()
    cache = empty_pool(m, 1, 1, 8, 128)
    kv = x.reshape(1, 1, 8, 128).cuda()
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, kv, -kv, zero, zero[0], dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for (codes, e), v in zip(pool_values(cache), (x, -x)):
        wc, we = C.quantise(f64(v))
        np.testing.assert_array_equal(codes[0, 0], wc)
        np.testing.assert_array_equal(e[0, 0], we)


def test_non_finite_values_are_reported_and_stored_as_numbers():
    m = sfa()
    x = torch.ones(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1, 3] = float("nan")
    x[0, 0, 2, 40] = float("-inf")
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for lens, want in ((1, 0), (2, m.SFA_ERR_INVALID_ARG), (4, m.SFA_ERR_INVALID_ARG)):
        cache = empty_pool(m, 1, 1, 4, 64)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.cache_write(cache, x, x, zero, zero[0], lens=torch.tensor([lens], dtype=torch.int32, device="cuda"),
                      dev_status=status)
        assert status.item() == want
    y = x.clone()
    y[0, 0, 1, 3] = 0.0
    y[0, 0, 2, 40] = -torch.finfo(torch.bfloat16).max
    wc, we = C.quantise(f64(y))
    for codes, e in pool_values(cache):
        np.testing.assert_array_equal(codes[0], wc[0])
        np.testing.assert_array_equal(e[0], we[0])


@pytest.mark.parametrize("what", ["page", "negative page", "behind", "before"])
def test_tokens_without_a_place_are_reported_and_skipped(what):
    case = (2, 3, 20, 64, 8, False, False, "bhld")
    m, cache, k, v, table, start, lens = _write_setup(case)
    start[:] = 0
    bad = []  # (batch, tokens that have no place)
    if what == "page":
        table[1, 0, 1] = cache.k.shape[0]
        bad = range(8, 16)
    elif what == "negative page":
        table[1, 0, 1] = -1
        bad = range(8, 16)
    elif what == "behind":
        start[1] = 8 * table.shape[2] - 5
        bad = range(5, 20)
    else:
        start[1] = -3
        bad = range(0, 3)
    good = [i for i in range(20) if i not in bad]
    before = pool_values(cache)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, k, v, _gpu(table), _gpu(start), dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == m.SFA_ERR_BAD_SET
    for (codes, e), (wc, we), x in zip(pool_values(cache), before, (f64(k), f64(v))):
        c_new, e_new = C.quantise(x)
        for b in range(2):
            for h in range(3):
                for i in (range(20) if b == 0 else good):
                    at = C.place(table, 3, 8, b, h, int(start[b]) + i)
                    wc[at], we[at] = c_new[b, h, i], e_new[b, h, i]
        np.testing.assert_array_equal(codes, wc)
        np.testing.assert_array_equal(e, we)
    status.zero_()
    ko = torch.full_like(k, 5.0)
    vo = torch.full_like(v, 5.0)
    m.cache_read(cache, _gpu(table), _gpu(start), 20, k_out=ko, v_out=vo, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == m.SFA_ERR_BAD_SET
    assert (ko[1][:, list(bad)] == 5).all()
    np.testing.assert_array_equal(f64(ko[1][:, good]), C.dequantise(*C.quantise(f64(k)))[1][:, good])


APPEND_CASES = [
    (1, 1, 1, 1, 128, 1, False, False, "half", (128,)),
    (3, 6, 2, 1, 64, 16, False, False, "half", (32,)),
    (2, 6, 3, 41, 128, 7, True, True, "interleaved", (44, 42, 42)),
    (1, 12, 12, 333, 64, 40, True, False, "interleaved", (22,)),
    (2, 80, 40, 33, 64, 16, False, True, "half", (48,)),
    # a warp for every token, and more heads than it looks up at a time
    (2, 40, 40, 1250, 64, 16, False, True, "half", (64,)),
    (1, 2, 35, 2400, 128, 24, True, False, "interleaved", (64, 32)),
    # several tokens a warp
    (3, 3, 1, 1777, 64, 40, True, True, "half", (32,)),
    (1, 1, 1, 5001, 128, 16, False, False, "interleaved", (44, 42, 42)),
    (7, 4, 3, 701, 128, 1560, True, True, "half", (128,)),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: f"B{c[0]}H{c[1]}.{c[2]}L{c[3]}d{c[4]}P{c[5]}")
def test_append_is_norm_rope_then_write(case):
    B, H, Hk, L, d, P, per_head, ragged, layout, axes = case
    m, cache, k, v, table, start, lens = _write_setup((B, Hk, L, d, P, per_head, ragged, "blhd"))
    g = np.random.default_rng(L)
    q = torch.from_numpy(g.standard_normal((B, H, L, d))).bfloat16().cuda()
    w = torch.from_numpy(1 + 0.2 * g.standard_normal((2, d))).float().cuda()
    args = dict(rope=m.rope_table(axes), positions=_positions(g, B, L, len(axes), True).cuda(), q_weight=w[0],
                k_weight=w[1], layout=layout)
    other = m.FrameCache(*(t.clone() for t in cache))
    q_out = torch.full_like(q, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = m.cache_append(cache, q, k, v, _gpu(table), _gpu(start), lens=_gpu(lens), q_out=q_out, dev_status=status, **args)
    yq, yk = m.qk_norm_rope(q, k, **args)
    m.cache_write(other, yk, v, _gpu(table), _gpu(start), lens=_gpu(lens))
    torch.cuda.synchronize()
    assert status.item() == 0 and got is q_out
    for x, y in zip(cache, other):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for b in range(B):
        n = L if lens is None else int(lens[b])
        assert torch.equal(q_out[b, :, :n], yq[b, :, :n]) and (q_out[b, :, n:] == 5).all()


def test_last_writer_of_chunks_in_order():
    """Chunk after chunk into a per-head ring of frames: the table decides which page a frame
    overwrites, and every head keeps its own."""
    m, g = sfa(), np.random.default_rng(5)
    P, Hk, d = 24, 2, 64
    cache = m.cache_create(5, P, d)
    ring = [[0, 1], [2, 3, 4]]  # head 0 keeps 2 frames, head 1 keeps 3
    frames = []
    for t in range(4):
        k = torch.from_numpy(g.standard_normal((1, Hk, P, d))).bfloat16().cuda()
        frames.append(k)
        table = torch.tensor([[[ring[h][t % len(ring[h])]] for h in range(Hk)]], dtype=torch.int32, device="cuda")
        m.cache_write(cache, k, k, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    for h, want in ((0, [2, 3]), (1, [1, 2, 3])):
        table = torch.tensor([[ring[h][t % len(ring[h])] for t in want]], dtype=torch.int32, device="cuda")
        ko, _ = m.cache_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), P * len(want))
        back = np.concatenate([C.dequantise(*C.quantise(f64(frames[t][0, h]))) for t in want])
        np.testing.assert_array_equal(f64(ko[0, 0]), back)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the last page is written and read, the first one is not."""
    m = sfa()
    P, d = 4096, 128
    n_pages = (1 << 32) // (P * d) + 4
    cache = m.cache_create(n_pages, P, d)
    x = torch.randn(1, 1, P, d, device="cuda").bfloat16()
    table = torch.tensor([[0, n_pages - 1]], dtype=torch.int32, device="cuda")
    start = torch.tensor([P], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_write(cache, x, x, table, start, dev_status=status)
    ko, vo = m.cache_read(cache, table, start, P, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    np.testing.assert_array_equal(f64(ko), C.dequantise(*C.quantise(f64(x))))
    assert torch.equal(ko, vo) and (cache.k[0].view(torch.uint8) == 0).all()


def test_other_stream_and_graph_replay():
    m, cache, k, v, table, start, lens = _write_setup((2, 3, 19, 64, 8, False, False, "bhld"))
    t, s = _gpu(table), _gpu(start)
    ref = m.FrameCache(*(x.clone() for x in cache))
    m.cache_write(ref, k, v, t, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        m.cache_write(cache, k, v, t, s)
    side.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(cache, ref))
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.cache_write(cache, k, v, t, s)
        m.cache_read(cache, t, s, 19, k_out=ko, v_out=vo)
    k.copy_(torch.randn_like(k))  # a replay reads what the tensors hold then
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(ko), C.dequantise(*C.quantise(f64(k))))
    np.testing.assert_array_equal(f64(vo), C.dequantise(*C.quantise(f64(v))))
