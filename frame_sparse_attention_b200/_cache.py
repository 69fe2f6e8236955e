"""Binding of the 8-bit frame cache: norm and rotation of new queries and keys, writing and
reading the cache, and attention over it (sfa_qk_norm_rope, sfa_cache_write,
sfa_cache_append, sfa_cache_read, sfa_forward_cache in include/sfa.h).

Like the rest of the binding it only marshals tensors; every call runs on the tensors'
device, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from ._lib import _check, _require, load

CACHE_BLOCK = 32  # elements of a cached row that share a scale
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_MAX_AXES = 4

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class CacheDesc(ctypes.Structure):
    """sfa_cache."""
    _fields_ = [("n_pages", _i32), ("heads", _i32), ("page_len", _i32), ("d", _i32), ("k", _vp), ("v", _vp),
                ("k_scale", _vp), ("v_scale", _vp), ("table", _vp), ("table_len", _i32),
                ("table_stride_b", _i64), ("table_stride_h", _i64)]


class RopeDesc(ctypes.Structure):
    """sfa_rope."""
    _fields_ = [("inv_freq", _vp), ("positions", _vp), ("pos_stride_b", _i64), ("pos_stride_t", _i64),
                ("layout", _i32), ("n_axes", _i32), ("axis_pairs", _i32 * ROPE_MAX_AXES), ("scale", _f32)]


class RowsDesc(ctypes.Structure):
    """sfa_rows_desc (each stride array as its three entries)."""
    _fields_ = [("B", _i32), ("H", _i32), ("H_kv", _i32), ("L", _i32), ("d", _i32), ("eps", _f32)] + \
               [(f"{t}_stride{i}", _i64) for t in ("q", "k", "v", "q_out", "k_out", "v_out") for i in range(3)] + \
               [("start_stride_b", _i64), ("start_stride_h", _i64)]


class CacheAttnDesc(ctypes.Structure):
    """sfa_cache_attn_desc."""
    _fields_ = [("B", _i32), ("H", _i32), ("H_kv", _i32), ("Lq", _i32), ("d", _i32), ("scale", _f32), ("causal", _i32),
                ("max_kv", _i32)] + \
               [(f"{t}_stride{i}", _i64) for t in ("q", "o") for i in range(3)] + \
               [("len_stride_b", _i64), ("len_stride_h", _i64), ("timeout_us", ctypes.c_uint32),
                ("debug_flags", ctypes.c_uint32)]


class RopeTable(NamedTuple):
    """Rotary frequencies: inv_freq float64 [R/2] on the GPU, the pairs of each position axis
    (they add up to R/2), and the factor that long-context scalings put on rotated values."""
    inv_freq: torch.Tensor
    axis_pairs: tuple
    scale: float = 1.0


class FrameCache(NamedTuple):
    """An 8-bit page pool: codes float8_e4m3fn [n_pages, heads, page_len, d] and scales
    float8_e8m0fnu [n_pages, heads, page_len, d/32] of the keys and the values.  heads is the
    number of key heads, or 1 for pages that belong to one head each (then every head has its
    own row of the page table and can keep other frames than its neighbours)."""
    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor


def cache_create(n_pages: int, page_len: int, d: int, heads: int = 1, device="cuda") -> FrameCache:
    """An empty page pool (zeros).  Size: 2 (d + d/32) bytes per row of a page."""
    _require(d in (64, 128), "expected d in (64, 128)")
    shape = (int(n_pages), int(heads), int(page_len))

    def codes():
        return torch.zeros(shape + (d,), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)

    def scales():
        return torch.full(shape + (d // CACHE_BLOCK,), 127, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
    return FrameCache(codes(), scales(), codes(), scales())


def rope_table(axis_dims, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0, original_len: int = 0,
               beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda") -> RopeTable:
    """Frequencies theta^(-2i/n) of every axis (n = its rotated elements, even).

    scaling, for contexts ``factor`` times longer than trained: "linear" divides the
    frequencies by factor; "ntk" raises theta to theta * factor^(n/(n-2)); "yarn" (Peng et al.
    2023) divides those that turn less than beta_slow times over ``original_len`` positions,
    keeps those that turn more than beta_fast times, blends the ones between, and scales
    rotated values by 0.1 ln(factor) + 1."""
    dims = [int(n) for n in axis_dims]
    _require(0 < len(dims) <= ROPE_MAX_AXES and all(n >= 0 and n % 2 == 0 for n in dims) and sum(dims) > 0,
             "expected 1 to 4 even axis dimensions")
    _require(scaling in ("none", "linear", "ntk", "yarn"), "expected scaling in (none, linear, ntk, yarn)")
    _require(factor > 0 and theta > 0, "expected factor > 0 and theta > 0")
    _require(scaling != "yarn" or original_len > 0, "yarn needs original_len")
    freq, scale = [], 1.0
    for n in dims:
        base = theta * factor ** (n / (n - 2)) if scaling == "ntk" and n > 2 else theta
        for i in range(n // 2):
            f = base ** (-2.0 * i / n)
            if scaling == "linear":
                f /= factor
            elif scaling == "yarn":
                turns = original_len * f / (2.0 * math.pi)
                keep = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
                f = keep * f + (1.0 - keep) * f / factor
            freq.append(f)
    if scaling == "yarn" and factor > 1.0:
        scale = 0.1 * math.log(factor) + 1.0
    return RopeTable(torch.tensor(freq, dtype=torch.float64, device=device), tuple(n // 2 for n in dims), scale)


# ---------------------------------------------------------------- marshalling
def _launch(device, fn, args, stream, what):
    """fn(*args, stream) with ``device`` current."""
    if device.type != "cuda":
        raise ValueError(f"{what}: expected CUDA tensors")
    index = device.index
    if index == torch.cuda.current_device():
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            if stream is None:
                stream = torch.cuda.current_stream().cuda_stream
            elif not isinstance(stream, int):
                stream = stream.cuda_stream
            status = fn(*args, stream)
    if status:
        _check(status, what)


def _rows(name, t, device, shape=None):
    if t.dtype != torch.bfloat16 or t.device != device or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a bf16 tensor [B, H, L, d] on {device} with d contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")


def _ints(name, t, device, shapes):
    if t.dtype != torch.int32 or t.device != device or tuple(t.shape) not in shapes:
        raise ValueError(f"{name} must be an int32 tensor on {device} of shape {' or '.join(map(str, shapes))}")


def _check_status(dev_status, device):
    if dev_status is not None:
        _require(dev_status.dtype == torch.int32 and dev_status.device == device and dev_status.numel() >= 1,
                 f"dev_status must be an int32 tensor on {device}")
        return dev_status.data_ptr()
    return None


def _per_head(name, t, device, B, H_kv):
    """(batch stride, head stride) of an int32 tensor [B] or [B, H_kv]."""
    _ints(name, t, device, ((B,), (B, H_kv), (B, 1)))
    return t.stride(0), (t.stride(1) if t.dim() == 2 and t.shape[1] > 1 else 0)


def _lens(lens, device, B):
    if lens is None:
        return None
    _ints("lens", lens, device, ((B,),))
    _require(lens.is_contiguous(), "expected lens.is_contiguous()")
    return lens.data_ptr()


def _weight(name, w, device, d):
    if w is None:
        return None
    if w.dtype != torch.float32 or w.device != device or tuple(w.shape) != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor [{d}] on {device}")
    return w.data_ptr()


def _cache_desc(cache, table, device, B, H_kv, d):
    k, ks, v, vs = cache.k, cache.k_scale, cache.v, cache.v_scale
    shape = tuple(k.shape)
    _require(len(shape) == 4 and shape[3] == d, f"expected cache codes [n_pages, heads, page_len, {d}]")
    s_shape = shape[:3] + (d // CACHE_BLOCK,)
    for name, t, want, dtype in (("k", k, shape, torch.float8_e4m3fn), ("v", v, shape, torch.float8_e4m3fn),
                                 ("k_scale", ks, s_shape, torch.float8_e8m0fnu),
                                 ("v_scale", vs, s_shape, torch.float8_e8m0fnu)):
        if t.dtype != dtype or t.device != device or tuple(t.shape) != want or not t.is_contiguous():
            raise ValueError(f"cache.{name} must be a contiguous {dtype} tensor {want} on {device}")
    _require(table.dtype == torch.int32 and table.device == device and table.dim() in (2, 3) and table.stride(-1) == 1,
             f"table must be an int32 tensor [B, N] or [B, H_kv, N] on {device}")
    rows = table.shape[1] if table.dim() == 3 else 1
    _require(table.shape[0] == B and rows in (1, H_kv), f"expected table [{B}, {H_kv} or 1, N]")
    return CacheDesc(shape[0], shape[1], shape[2], d, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                     table.data_ptr(), table.shape[-1], table.stride(0), table.stride(1) if rows > 1 else 0)


def _rope_desc(rope, positions, layout, device, B, L):
    """A pointer to the sfa_rope of this call, or None."""
    if rope is None:
        return None
    f, pairs = rope.inv_freq, rope.axis_pairs
    if f.dtype != torch.float64 or f.device != device or not f.is_contiguous() or f.numel() != sum(pairs):
        raise ValueError(f"rope.inv_freq must be a contiguous float64 tensor [{sum(pairs)}] on {device}")
    _require(layout in ROPE_LAYOUTS, "expected layout 'interleaved' or 'half'")
    n = len(pairs)
    _require(0 < n <= ROPE_MAX_AXES, "expected 1 to 4 position axes")
    _require(positions is not None, "rope needs positions")
    _ints("positions", positions, device, ((B, L, n), (1, L, n), (L, n)))
    _require(n == 1 or positions.stride(-1) == 1, "expected positions with the axes contiguous")
    sb = positions.stride(0) if positions.dim() == 3 and positions.shape[0] == B else 0
    r = RopeDesc(f.data_ptr(), positions.data_ptr(), sb, positions.stride(-2), ROPE_LAYOUTS[layout], n)
    r.scale = rope.scale
    for i, p in enumerate(pairs):
        r.axis_pairs[i] = p
    return ctypes.byref(r)


_NO = (0, 0, 0)


def qk_norm_rope(q, k=None, rope: RopeTable | None = None, positions=None, q_weight=None, k_weight=None,
                 eps: float | None = 1e-6, layout: str = "interleaved", q_out=None, k_out=None, stream=None):
    """RMS norm of every head's query and key row and their rotary positions, in one pass.

    q bf16 [B, H, L, d], k bf16 [B, H_kv, L, d] (either may be None); weights fp32 [d] or None
    (ones); eps None: no norm.  rope None: no rotation, else positions int32 [B, L, axes]
    (or [L, axes], shared by the batch).  Returns (q_out, k_out), bf16, None where there was no
    input; an output may be its input (in place)."""
    t = q if q is not None else k
    _require(t is not None, "qk_norm_rope needs q or k")
    device = t.device
    _require(t.dim() == 4, "expected tensors [B, H, L, d]")
    B, _, L, d = t.shape
    H, H_kv, sq, so, sk, sko = 0, 0, _NO, _NO, _NO, _NO
    qp = qop = kp = kop = None
    if q is not None:
        _rows("q", q, device)
        q_out = torch.empty_like(q) if q_out is None else q_out
        _rows("q_out", q_out, device, q.shape)
        H, sq, so, qp, qop = q.shape[1], q.stride(), q_out.stride(), q.data_ptr(), q_out.data_ptr()
    if k is not None:
        _rows("k", k, device, (B, k.shape[1], L, d))
        k_out = torch.empty_like(k) if k_out is None else k_out
        _rows("k_out", k_out, device, k.shape)
        H_kv, sk, sko, kp, kop = k.shape[1], k.stride(), k_out.stride(), k.data_ptr(), k_out.data_ptr()
    desc = RowsDesc(B, H, H_kv, L, d, -1.0 if eps is None else eps, *sq[:3], *sk[:3], *_NO, *so[:3], *sko[:3])
    _launch(device, load().sfa_qk_norm_rope,
            (ctypes.byref(desc), _rope_desc(rope, positions, layout, device, B, L), qp, kp,
             _weight("q_weight", q_weight, device, d), _weight("k_weight", k_weight, device, d), qop, kop),
            stream, "sfa_qk_norm_rope")
    return q_out if q is not None else None, k_out if k is not None else None


def cache_write(cache: FrameCache, k, v, table, start, lens=None, dev_status=None, stream=None):
    """Write new keys and values bf16 [B, H_kv, L, d] into the cache: token i of (b, h) becomes
    logical token start[b][h] + i.  table int32 [B, N] or [B, H_kv, N] of page numbers, start
    int32 [B] or [B, H_kv], lens int32 [B] (rows from there on are padding) or None."""
    device = k.device
    _rows("k", k, device)
    _rows("v", v, device, k.shape)
    B, H_kv, L, d = k.shape
    cd = _cache_desc(cache, table, device, B, H_kv, d)
    desc = RowsDesc(B, 0, H_kv, L, d, -1.0, *_NO, *k.stride()[:3], *v.stride()[:3], *_NO, *_NO, *_NO,
                    *_per_head("start", start, device, B, H_kv))
    _launch(device, load().sfa_cache_write,
            (ctypes.byref(desc), ctypes.byref(cd), k.data_ptr(), v.data_ptr(), start.data_ptr(),
             _lens(lens, device, B), _check_status(dev_status, device)), stream, "sfa_cache_write")


def cache_append(cache: FrameCache, q, k, v, table, start, lens=None, rope: RopeTable | None = None, positions=None,
                 q_weight=None, k_weight=None, eps: float | None = 1e-6, layout: str = "interleaved", q_out=None,
                 dev_status=None, stream=None):
    """qk_norm_rope of q and k, and cache_write of those keys and v, in one pass (the bf16 keys
    are not written).  Arguments as theirs; returns q_out.  Padding rows of q_out (from lens[b]
    on) are left as they are."""
    device = q.device
    _rows("q", q, device)
    B, H, L, d = q.shape
    _rows("k", k, device, (B, k.shape[1], L, d))
    _rows("v", v, device, k.shape)
    H_kv = k.shape[1]
    q_out = torch.empty_like(q) if q_out is None else q_out
    _rows("q_out", q_out, device, q.shape)
    cd = _cache_desc(cache, table, device, B, H_kv, d)
    desc = RowsDesc(B, H, H_kv, L, d, -1.0 if eps is None else eps, *q.stride()[:3], *k.stride()[:3],
                    *v.stride()[:3], *q_out.stride()[:3], *_NO, *_NO, *_per_head("start", start, device, B, H_kv))
    _launch(device, load().sfa_cache_append,
            (ctypes.byref(desc), _rope_desc(rope, positions, layout, device, B, L), ctypes.byref(cd), q.data_ptr(),
             k.data_ptr(), v.data_ptr(), _weight("q_weight", q_weight, device, d),
             _weight("k_weight", k_weight, device, d), q_out.data_ptr(), start.data_ptr(), _lens(lens, device, B),
             _check_status(dev_status, device)), stream, "sfa_cache_append")
    return q_out


def cache_read(cache: FrameCache, table, start, L: int, lens=None, k_out=None, v_out=None, H_kv: int | None = None,
               dev_status=None, stream=None):
    """Logical tokens start[b][h] + i, i < min(L, lens[b]), of every (b, h) back as bf16
    [B, H_kv, L, d]: (k_out, v_out).  Other rows are left as they are (zero where the outputs
    are allocated here).  H_kv: key heads, where neither the pool nor the table says so."""
    device = cache.k.device
    _require(cache.k.dim() == 4 and table.dim() in (2, 3), "expected cache codes [n_pages, heads, page_len, d]")
    B, d = table.shape[0], cache.k.shape[3]
    if H_kv is None:
        H_kv = k_out.shape[1] if k_out is not None else max(cache.k.shape[1], table.shape[1] if table.dim() == 3 else 1)
    shape = (B, H_kv, int(L), d)
    k_out = torch.zeros(shape, dtype=torch.bfloat16, device=device) if k_out is None else k_out
    v_out = torch.zeros(shape, dtype=torch.bfloat16, device=device) if v_out is None else v_out
    _rows("k_out", k_out, device, shape)
    _rows("v_out", v_out, device, shape)
    cd = _cache_desc(cache, table, device, B, H_kv, d)
    desc = RowsDesc(B, 0, H_kv, int(L), d, -1.0, *_NO, *_NO, *_NO, *_NO, *k_out.stride()[:3], *v_out.stride()[:3],
                    *_per_head("start", start, device, B, H_kv))
    _launch(device, load().sfa_cache_read,
            (ctypes.byref(desc), ctypes.byref(cd), start.data_ptr(), _lens(lens, device, B), k_out.data_ptr(),
             v_out.data_ptr(), _check_status(dev_status, device)), stream, "sfa_cache_read")
    return k_out, v_out


def _attn(q, cache, table, kv_lens, causal, max_kv, scale, out, H_kv, timeout_us=0, debug_flags=0):
    device = q.device
    B, H, Lq, d = q.shape
    if H_kv is None:
        H_kv = max(cache.k.shape[1], table.shape[1] if table.dim() == 3 else 1,
                   kv_lens.shape[1] if kv_lens.dim() == 2 else 1)
    cd = _cache_desc(cache, table, device, B, H_kv, d)
    desc = CacheAttnDesc(B, H, H_kv, Lq, d, 1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0, max_kv,
                         *q.stride()[:3], *out.stride()[:3], *_per_head("kv_lens", kv_lens, device, B, H_kv),
                         timeout_us, debug_flags)
    return desc, cd


def forward_cache_workspace_bytes(q, cache: FrameCache, table, kv_lens, max_kv: int = 0, H_kv: int | None = None) -> int:
    """Device workspace bytes of forward_cache for these shapes."""
    desc, cd = _attn(q, cache, table, kv_lens, False, max_kv, None, q, H_kv)
    out = ctypes.c_size_t(0)
    _check(load().sfa_forward_cache_workspace(ctypes.byref(desc), ctypes.byref(cd), ctypes.byref(out)),
           "sfa_forward_cache_workspace")
    return out.value


def forward_cache(q, cache: FrameCache, table, kv_lens, causal: bool = False, q_lens=None, max_kv: int = 0,
                  scale: float | None = None, out=None, lse=None, workspace=None, H_kv: int | None = None,
                  dev_status=None, stream=None, timeout_us: int = 0, debug_flags: int = 0):
    """Attention of new tokens over the cache: (O bf16 like q, LSE fp32 [B, H, Lq]).

    q bf16 [B, H, Lq, d]; kv_lens int32 [B] or [B, H_kv]: logical tokens [0, n) are the keys and
    values.  q_lens int32 [B]: rows from there on are padding, left as they are.  causal: the
    rows are the last of the n tokens and see none behind themselves.  max_kv: an upper bound of
    kv_lens, for the split of the work (0: all that the table can hold).  workspace: a uint8
    tensor of forward_cache_workspace_bytes (allocated here when not given).  H_kv: key heads,
    where neither the pool, the table nor kv_lens says so.  Rows that see no key give O = 0,
    LSE = -inf, so the result merges with other branches by lse_merge."""
    device = q.device
    _rows("q", q, device)
    B, H, Lq, d = q.shape
    out = torch.empty_like(q) if out is None else out
    _rows("out", out, device, q.shape)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=device)
    elif lse.dtype != torch.float32 or lse.device != device or tuple(lse.shape) != (B, H, Lq) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 tensor {(B, H, Lq)} on {device}")
    desc, cd = _attn(q, cache, table, kv_lens, causal, max_kv, scale, out, H_kv, timeout_us, debug_flags)
    lib = load()
    if workspace is None:
        need = ctypes.c_size_t(0)
        _check(lib.sfa_forward_cache_workspace(ctypes.byref(desc), ctypes.byref(cd), ctypes.byref(need)),
               "sfa_forward_cache_workspace")
        if need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _launch(device, lib.sfa_forward_cache,
            (ctypes.byref(desc), ctypes.byref(cd), q.data_ptr(), kv_lens.data_ptr(), _lens(q_lens, device, B),
             out.data_ptr(), lse.data_ptr(), ws, ws_bytes, _check_status(dev_status, device)), stream,
            "sfa_forward_cache")
    return out, lse
