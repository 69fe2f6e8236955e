"""Refusals of the 8-bit frame cache calls: on the host, before any launch (CPU)."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def sfa():
    import os

    import frame_sparse_attention_b200 as sfa
    from frame_sparse_attention_b200 import build
    if not os.path.exists(build.LIB):
        build.build()
    sfa.load()
    return sfa


GOOD = 1 << 20  # an aligned address that no accepted call would survive using


_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class CacheDesc(ctypes.Structure):  # sfa_cache
    _fields_ = [("n_pages", _i32), ("heads", _i32), ("page_len", _i32), ("d", _i32), ("k", _vp), ("v", _vp),
                ("k_scale", _vp), ("v_scale", _vp), ("table", _vp), ("table_len", _i32),
                ("table_stride_b", _i64), ("table_stride_h", _i64)]


class RopeDesc(ctypes.Structure):  # sfa_rope
    _fields_ = [("inv_freq", _vp), ("positions", _vp), ("pos_stride_b", _i64), ("pos_stride_t", _i64),
                ("layout", _i32), ("n_axes", _i32), ("axis_pairs", _i32 * 4), ("scale", _f32)]


class RowsDesc(ctypes.Structure):  # sfa_rows_desc
    _fields_ = [("B", _i32), ("H", _i32), ("H_kv", _i32), ("L", _i32), ("d", _i32), ("eps", _f32)] + \
               [(f"{t}_stride{i}", _i64) for t in ("q", "k", "v", "q_out", "k_out", "v_out") for i in range(3)] + \
               [("start_stride_b", _i64), ("start_stride_h", _i64)]


class CacheAttnDesc(ctypes.Structure):  # sfa_cache_attn_desc
    _fields_ = [("B", _i32), ("H", _i32), ("H_kv", _i32), ("Lq", _i32), ("d", _i32), ("scale", _f32), ("causal", _i32),
                ("max_kv", _i32)] + \
               [(f"{t}_stride{i}", _i64) for t in ("q", "o") for i in range(3)] + \
               [("len_stride_b", _i64), ("len_stride_h", _i64), ("timeout_us", ctypes.c_uint32),
                ("debug_flags", ctypes.c_uint32)]


def test_the_bindings_structs_have_cs_sizes(sfa):
    from frame_sparse_attention_b200 import _cache as c
    for packed, struct in ((c._CACHE, CacheDesc), (c._ROPE, RopeDesc), (c._ROWS, RowsDesc), (c._ATTN, CacheAttnDesc)):
        assert packed.size == ctypes.sizeof(struct)


def _structs():
    rows = RowsDesc(2, 4, 2, 8, 64, 1e-6)
    for t, heads in (("q", 4), ("k", 2), ("v", 2), ("q_out", 4), ("k_out", 2), ("v_out", 2)):
        for i, s in enumerate((heads * 8 * 64, 8 * 64, 64)):
            setattr(rows, f"{t}_stride{i}", s)
    rows.start_stride_b = 1
    cache = CacheDesc(4, 2, 16, 64, GOOD, GOOD, GOOD, GOOD, GOOD, 3, 3, 0)
    rope = RopeDesc(GOOD, GOOD, 8, 1, 0, 1)
    rope.axis_pairs[0] = 16
    rope.scale = 1.0
    return rows, cache, rope


def _call(sfa, fn, rows, cache, rope, p=GOOD):
    lib, r = sfa.load(), ctypes.byref
    rp = None if rope is None else r(rope)
    rows = None if rows is None else r(rows)
    cp = None if cache is None else r(cache)
    if fn == "norm":
        return lib.sfa_qk_norm_rope(rows, rp, p, p, None, None, p, p, None)
    if fn == "write":
        return lib.sfa_cache_write(rows, cp, p, p, GOOD, None, None, None)
    if fn == "append":
        return lib.sfa_cache_append(rows, rp, cp, p, p, p, None, None, p, GOOD, None, None, None)
    return lib.sfa_cache_read(rows, cp, GOOD, None, p, p, None, None)


ALL = ("norm", "write", "append", "read")
CACHE = ("write", "append", "read")


@pytest.mark.parametrize("over,code", [(dict(B=-1), 1), (dict(L=-1), 1), (dict(d=96), 2), (dict(d=32), 2),
                                       (dict(H_kv=0), 1), (dict(H_kv=2000), 1)])
@pytest.mark.parametrize("fn", ALL)
def test_shapes(sfa, fn, over, code):
    rows, cache, rope = _structs()
    for k, v in over.items():
        setattr(rows, k, v)
    assert _call(sfa, fn, rows, cache, rope) == code
    assert _call(sfa, fn, None, cache, rope) == 1


@pytest.mark.parametrize("over", [dict(eps=float("nan")), dict(eps=float("inf"))])
@pytest.mark.parametrize("fn", ("norm", "append"))
def test_eps(sfa, fn, over):
    rows, cache, rope = _structs()
    rows.eps = over["eps"]
    assert _call(sfa, fn, rows, cache, rope) == 1


@pytest.mark.parametrize("fn", ALL)
def test_addresses_and_strides(sfa, fn):
    rows, cache, rope = _structs()
    assert _call(sfa, fn, rows, cache, rope, p=GOOD + 2) == 1
    assert _call(sfa, fn, rows, cache, rope, p=None) == 1
    for t in {"norm": ("q", "k", "q_out", "k_out"), "write": ("k", "v"), "append": ("q", "k", "v", "q_out"),
              "read": ("k_out", "v_out")}[fn]:
        for i, bad in ((0, 0), (1, 12), (2, -64), (2, 1 << 40)):
            rows, cache, rope = _structs()
            setattr(rows, f"{t}_stride{i}", bad)
            assert _call(sfa, fn, rows, cache, rope) == 1, (t, i, bad)


@pytest.mark.parametrize("over,code", [
    (dict(n_pages=0), 1), (dict(heads=3), 1), (dict(page_len=0), 1), (dict(d=128), 1), (dict(d=48), 2), (dict(k=None), 1),
    (dict(v_scale=None), 1), (dict(table=None), 1), (dict(k=GOOD + 8), 1), (dict(k_scale=GOOD + 1), 1), (dict(table_len=0), 1),
    (dict(table_stride_b=-1), 1), (dict(table_len=1 << 20, page_len=1 << 12), 1)])
@pytest.mark.parametrize("fn", CACHE)
def test_cache(sfa, fn, over, code):
    rows, cache, rope = _structs()
    for k, v in over.items():
        setattr(cache, k, v)
    assert _call(sfa, fn, rows, cache, rope) == code
    assert _call(sfa, fn, rows, None, rope) == 1


@pytest.mark.parametrize("fn", CACHE)
def test_start(sfa, fn):
    rows, cache, rope = _structs()
    rows.start_stride_h = -1
    assert _call(sfa, fn, rows, cache, rope) == 1


@pytest.mark.parametrize("fn", ("write", "append"))
def test_heads_that_would_meet_in_one_place(sfa, fn):
    rows, cache, rope = _structs()
    cache.heads = 1
    cache.table_stride_h = 0
    assert _call(sfa, fn, rows, cache, rope) == 1
    rows.H_kv, rows.B = 1, 0  # (nothing to do, so that nothing is launched)
    assert _call(sfa, fn, rows, cache, rope) == 0


@pytest.mark.parametrize("over,pairs,code", [
    (dict(inv_freq=None), (16,), 1), (dict(positions=None), (16,), 1), (dict(inv_freq=GOOD + 4), (16,), 1),
    (dict(positions=GOOD + 2), (16,), 1), (dict(layout=2), (16,), 1), (dict(n_axes=0), (), 1), (dict(n_axes=5), (), 1),
    (dict(scale=float("nan")), (16,), 1), (dict(pos_stride_t=-1), (16,), 1), (dict(), (0,), 1), (dict(), (33,), 1),
    (dict(n_axes=2), (20, 20), 1), (dict(n_axes=2), (-1, 20), 1), (dict(layout=1), (12,), 2)])
@pytest.mark.parametrize("fn", ("norm", "append"))
def test_rope(sfa, fn, over, pairs, code):
    rows, cache, rope = _structs()
    for k, v in over.items():
        setattr(rope, k, v)
    for i, p in enumerate(pairs):
        rope.axis_pairs[i] = p
    assert _call(sfa, fn, rows, cache, rope) == code


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("dim", ("B", "L"))
def test_nothing_to_do(sfa, fn, dim):
    rows, cache, rope = _structs()
    setattr(rows, dim, 0)
    assert _call(sfa, fn, rows, cache, rope, p=None) == 0


def test_norm_rope_needs_an_input_and_its_output(sfa):
    lib, (rows, _, _) = sfa.load(), _structs()
    r = ctypes.byref(rows)
    assert lib.sfa_qk_norm_rope(r, None, None, None, None, None, None, None, None) == 1
    assert lib.sfa_qk_norm_rope(r, None, GOOD, None, None, None, None, None, None) == 1
    assert lib.sfa_qk_norm_rope(r, None, GOOD, None, None, None, GOOD, GOOD, None) == 1


def test_weights_are_aligned(sfa):
    lib, r = sfa.load(), ctypes.byref
    rows, cache, rope = _structs()
    for w in ((GOOD + 4, None), (None, GOOD + 8)):
        assert lib.sfa_qk_norm_rope(r(rows), r(rope), GOOD, GOOD, *w, GOOD, GOOD, None) == 1
        assert lib.sfa_cache_append(r(rows), r(rope), r(cache), GOOD, GOOD, GOOD, *w, GOOD, GOOD, None, None, None) == 1


def test_binding_refuses_wrong_tensors(sfa):
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    cache = sfa.cache_create(4, 16, 64, heads=2, device="cpu")
    table, start = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        sfa.qk_norm_rope(q, k)
    with pytest.raises(ValueError):
        sfa.cache_write(cache, k, k, table, start)
    with pytest.raises(ValueError):
        sfa.cache_append(cache, q, k, k, table, start)
    with pytest.raises(ValueError):
        sfa.cache_read(cache, table, start, 8)
    bad = [dict(k=k.float()), dict(v=k[:, :1]), dict(table=table.long()), dict(table=table[:1]), dict(start=start[:1]),
           dict(start=start.long()), dict(lens=start.long()), dict(lens=torch.zeros(3, dtype=torch.int32)),
           dict(cache=sfa.cache_create(4, 16, 128, heads=2, device="cpu")),
           dict(cache=cache._replace(k_scale=cache.k_scale[..., :1])), dict(cache=cache._replace(k=k)),
           dict(k=k.transpose(2, 3))]
    for over in bad:
        a = dict(cache=cache, k=k, v=k, table=table, start=start, lens=None)
        a.update(over)
        with pytest.raises(ValueError):
            sfa.cache_write(**a)
    rope = sfa.rope_table((64,), device="cpu")
    pos = torch.zeros(2, 8, 1, dtype=torch.int32)
    for over in (dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:, :7]), dict(layout="other"),
                 dict(rope=rope._replace(inv_freq=rope.inv_freq.float())), dict(rope=rope._replace(axis_pairs=(16,))),
                 dict(q_weight=torch.ones(63)), dict(q_weight=torch.ones(64).double()), dict(q_out=k)):
        a = dict(rope=rope, positions=pos)
        a.update(over)
        with pytest.raises(ValueError):
            sfa.qk_norm_rope(q, k, **a)
    for args, kw in (((63,), {}), ((), {}), ((2,) * 5, {}), ((64,), dict(scaling="other")), ((64,), dict(factor=0.0)),
                     ((64,), dict(scaling="yarn", factor=2.0))):
        with pytest.raises(ValueError):
            sfa.rope_table(args, device="cpu", **kw)
    with pytest.raises(ValueError):
        sfa.cache_create(1, 1, 96, device="cpu")
    assert math.isclose(sfa.rope_table((8,), device="cpu").inv_freq[1].item(), 0.1)


def _attn(sfa):
    d = CacheAttnDesc(2, 4, 2, 8, 64, 0.125, 0, 0)
    for t in ("q", "o"):
        for i, s in enumerate((4 * 8 * 64, 8 * 64, 64)):
            setattr(d, f"{t}_stride{i}", s)
    d.len_stride_b = 1
    return d


def _attn_call(sfa, d, cache, q=GOOD, o=GOOD, lse=GOOD, lens=GOOD, ws=None, ws_bytes=0):
    r = ctypes.byref
    return sfa.load().sfa_forward_cache(None if d is None else r(d), None if cache is None else r(cache), q, lens, None, o,
                                        lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("over,code", [(dict(B=-1), 1), (dict(Lq=-1), 1), (dict(d=96), 2), (dict(H=0), 1), (dict(H=3), 1),
                                       (dict(H_kv=0), 1), (dict(H_kv=4), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
                                       (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(max_kv=-1), 1), (dict(len_stride_b=-1), 1),
                                       (dict(q_stride1=12), 1), (dict(o_stride2=0), 1), (dict(d=128), 1)])
def test_attention_descriptor(sfa, over, code):
    _, cache, _ = _structs()
    d = _attn(sfa)
    for k, v in over.items():
        setattr(d, k, v)
    assert _attn_call(sfa, d, cache) == code


def test_attention_addresses(sfa):
    _, cache, _ = _structs()
    d = _attn(sfa)
    assert _attn_call(sfa, None, cache) == 1 and _attn_call(sfa, d, None) == 1
    for k in ("q", "o", "lse", "lens"):
        assert _attn_call(sfa, d, cache, **{k: None}) == 1
    assert _attn_call(sfa, d, cache, q=GOOD + 8) == 1 and _attn_call(sfa, d, cache, o=GOOD + 2) == 1
    d.Lq = 0
    assert _attn_call(sfa, d, cache, q=None) == 0


def test_attention_workspace(sfa):
    _, cache, _ = _structs()
    d = _attn(sfa)
    cache.table_len, cache.page_len = 4096, 16  # 65536 tokens: the keys are cut into ranges
    need = ctypes.c_size_t(0)
    lib, r = sfa.load(), ctypes.byref
    assert lib.sfa_forward_cache_workspace(r(d), r(cache), r(need)) == 0 and need.value > 0 and need.value % 256 == 0
    assert _attn_call(sfa, d, cache) == 1                                           # none
    assert _attn_call(sfa, d, cache, ws=GOOD, ws_bytes=need.value - 1) == 1         # too small
    assert _attn_call(sfa, d, cache, ws=GOOD + 128, ws_bytes=need.value) == 1       # misaligned
    d.max_kv = 100
    assert lib.sfa_forward_cache_workspace(r(d), r(cache), r(need)) == 0 and need.value == 0
    assert lib.sfa_forward_cache_workspace(r(d), r(cache), None) == 1


def test_attention_binding_refuses_wrong_tensors(sfa):
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    cache = sfa.cache_create(4, 16, 64, heads=2, device="cpu")
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for over in (dict(), dict(q=q.float()), dict(kv_lens=lens.long()), dict(kv_lens=lens[:1]), dict(table=table.long()),
                 dict(out=q[:1]), dict(lse=torch.zeros(2, 4, 7)), dict(lse=torch.zeros(2, 4, 8).double()),
                 dict(q_lens=lens.long()), dict(H_kv=3), dict(q=q[..., :32]), dict(cache=cache._replace(v=cache.v[:2]))):
        a = dict(q=q, cache=cache, table=table, kv_lens=lens)
        a.update(over)
        with pytest.raises((ValueError, sfa.SfaError)):
            sfa.forward_cache(**a)


def test_binding_refuses_what_is_no_tensor_or_no_number(sfa):
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    cache = sfa.cache_create(4, 16, 64, heads=2, device="cpu")
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(q=q, cache=cache, table=table, kv_lens=lens)
    for over, error in ((dict(q=None), TypeError), (dict(table=[0]), TypeError), (dict(kv_lens=3), TypeError),
                        (dict(cache=cache[:3]), ValueError), (dict(cache=5), TypeError), (dict(max_kv=1 << 40), ValueError),
                        (dict(max_kv="8"), TypeError), (dict(timeout_us=-1), ValueError), (dict(debug_flags=1 << 32), ValueError),
                        (dict(scale="1"), TypeError), (dict(H_kv=1 << 35), ValueError), (dict(lse=0), TypeError),
                        (dict(stream=7), ValueError), (dict(kv_lens=torch.tensor(1, dtype=torch.int32)), ValueError),
                        (dict(table=torch.tensor(1, dtype=torch.int32)), ValueError), (dict(q=q[0]), ValueError)):
        with pytest.raises(error):
            sfa.forward_cache(**{**good, **over})
    rope = sfa.rope_table((64,), device="cpu")
    pos = torch.zeros(8, 1, dtype=torch.int32)
    for over, error in ((dict(rope=rope[:2]), ValueError), (dict(rope=3), TypeError), (dict(layout=None), ValueError),
                        (dict(rope=rope._replace(axis_pairs=())), ValueError), (dict(eps="1"), TypeError),
                        (dict(rope=rope._replace(axis_pairs=(8,) * 5)), ValueError), (dict(positions=3), TypeError),
                        (dict(q_weight=1.0), TypeError), (dict(q_out=1), TypeError)):
        with pytest.raises(error):
            sfa.qk_norm_rope(q, **{**dict(rope=rope, positions=pos), **over})
    with pytest.raises(ValueError):
        sfa.qk_norm_rope(None, None)
    for over, error in ((dict(L=-1), ValueError), (dict(L=1 << 31), ValueError), (dict(L=None), TypeError),
                        (dict(H_kv=0), ValueError), (dict(table=torch.tensor(1, dtype=torch.int32)), ValueError)):
        with pytest.raises(error):
            sfa.cache_read(**{**dict(cache=cache, table=table, start=lens, L=8), **over})
