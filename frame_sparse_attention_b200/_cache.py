"""Binding of the 8-bit frame cache: norm and rotation of new queries and keys, writing and
reading the cache, and attention over it (sfa_qk_norm_rope, sfa_cache_write,
sfa_cache_append, sfa_cache_read, sfa_forward_cache in include/sfa.h).

Like the rest of the binding it only marshals tensors; every call runs on the tensors'
device, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from ._lib import SfaError, _check, _require, load

CACHE_BLOCK = 32  # elements of a cached row that share a scale
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_MAX_AXES = 4

# The descriptors of include/sfa.h as native structs (field by field, C's padding written out)
_CACHE = struct.Struct("@4i5Pi4x2q")        # sfa_cache
_ROPE = struct.Struct("@2P2q6if4x")         # sfa_rope: inv_freq, positions, strides, layout, n_axes, axis_pairs, scale
_ROWS = struct.Struct("@5if18q2q")          # sfa_rows_desc: sizes, eps, q, k, v, q_out, k_out, v_out and start strides
_ATTN = struct.Struct("@5if2i6q2q2I")       # sfa_cache_attn_desc

_BF16, _I32, _F32, _F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


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
# These calls are a few microseconds of GPU time at a single token, so the checks below are
# written for few interpreter steps.
def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _launch(dev, fn, args, stream, what):
    """fn(*args, stream) with device ``dev`` current."""
    if dev < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    if stream is not None and not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == torch.cuda.current_device():
        status = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev) if stream is None else stream)
    if status:
        raise SfaError(status, what)


def _new(make, *args, stream, dev, **kw):
    """make(*args, **kw) for a call on ``stream``: what is allocated here belongs to that stream,
    whose order a fill and a later reuse of the memory then follow."""
    if stream is None:
        return make(*args, **kw)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _rows(name, t, dev, shape):
    """(strides, address) of a bf16 tensor of this shape."""
    if t.dtype is not _BF16 or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be a bf16 tensor {tuple(shape)} on device {dev}: {t.dtype} {tuple(t.shape)}")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name} must have d contiguous")
    return st[:3], t.data_ptr()


def _shape4(name, t):
    s = t.shape
    if len(s) != 4:
        raise ValueError(f"{name} must be [B, H, L, d]")
    return s


def _per_head(name, t, dev, B, H_kv):
    """(batch stride, head stride) of an int32 tensor [B], [B, 1] or [B, H_kv]."""
    s = t.shape
    if t.dtype is not _I32 or t.get_device() != dev or len(s) not in (1, 2) or s[0] != B or \
            (len(s) == 2 and s[1] != H_kv and s[1] != 1):
        raise ValueError(f"{name} must be an int32 tensor [{B}] or [{B}, {H_kv}] on device {dev}")
    st = t.stride()
    return (st[0], st[1]) if len(s) == 2 and s[1] > 1 else (st[0], 0)


def _lens(name, t, dev, B):
    if t is None:
        return None
    if t.dtype is not _I32 or t.get_device() != dev or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [{B}] on device {dev}")
    return t.data_ptr()


def _status(t, dev):
    if t is None:
        return None
    if t.dtype is not _I32 or t.get_device() != dev or t.numel() < 1:
        raise ValueError(f"dev_status must be an int32 tensor on device {dev}")
    return t.data_ptr()


def _weight(name, w, dev, d):
    if w is None:
        return None
    if w.dtype is not _F32 or w.get_device() != dev or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor [{d}] on device {dev}")
    return w.data_ptr()


def _cache_desc(cache, table, dev, B, H_kv, d):
    k, ks, v, vs = cache
    shape = k.shape
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"expected cache codes [n_pages, heads, page_len, {d}], have {tuple(shape)}")
    scales = (*shape[:3], d // CACHE_BLOCK)
    if k.dtype is not _E4M3 or v.dtype is not _E4M3 or ks.dtype is not _E8M0 or vs.dtype is not _E8M0 or \
            v.shape != shape or ks.shape != scales or vs.shape != scales:
        raise ValueError(f"expected a cache of float8_e4m3fn codes {tuple(shape)} and float8_e8m0fnu scales {scales}")
    if k.get_device() != dev or v.get_device() != dev or ks.get_device() != dev or vs.get_device() != dev or \
            not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError(f"expected a contiguous cache on device {dev}")
    ts, st = table.shape, table.stride()
    if table.dtype is not _I32 or table.get_device() != dev or len(ts) not in (2, 3) or ts[0] != B or \
            (ts[-1] > 1 and st[-1] != 1) or (len(ts) == 3 and ts[1] != 1 and ts[1] != H_kv):
        raise ValueError(f"table must be an int32 tensor [{B}, N] or [{B}, {H_kv}, N] on device {dev}, rows contiguous")
    return _CACHE.pack(*shape, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), table.data_ptr(), ts[-1],
                       st[0], st[1] if len(ts) == 3 and ts[1] > 1 else 0)


def _rope_desc(rope, positions, layout, dev, B, L):
    """The sfa_rope of this call, or None."""
    if rope is None:
        return None
    f, pairs, scale = rope
    n = len(pairs)
    if not 0 < n <= ROPE_MAX_AXES:
        raise ValueError(f"expected 1 to {ROPE_MAX_AXES} position axes")
    if f.dtype is not _F64 or f.get_device() != dev or f.shape != (sum(pairs),) or not f.is_contiguous():
        raise ValueError(f"rope.inv_freq must be a contiguous float64 tensor [{sum(pairs)}] on device {dev}")
    if layout not in ROPE_LAYOUTS:
        raise ValueError("expected layout 'interleaved' or 'half'")
    if positions is None:
        raise ValueError("rope needs positions")
    s, st = positions.shape, positions.stride()
    if positions.dtype is not _I32 or positions.get_device() != dev or len(s) not in (2, 3) or s[-1] != n or \
            s[-2] != L or (len(s) == 3 and s[0] != B and s[0] != 1) or (n > 1 and st[-1] != 1):
        raise ValueError(f"positions must be an int32 tensor [{B}, {L}, {n}] or [{L}, {n}] on device {dev}")
    return _ROPE.pack(f.data_ptr(), positions.data_ptr(), st[0] if len(s) == 3 and s[0] == B else 0, st[-2],
                      ROPE_LAYOUTS[layout], n, *pairs, *(0,) * (ROPE_MAX_AXES - n), scale)


_NO = (0, 0, 0)


def qk_norm_rope(q, k=None, rope: RopeTable | None = None, positions=None, q_weight=None, k_weight=None,
                 eps: float | None = 1e-6, layout: str = "interleaved", q_out=None, k_out=None, stream=None):
    """RMS norm of every head's query and key row and their rotary positions, in one pass.

    q bf16 [B, H, L, d], k bf16 [B, H_kv, L, d] (either may be None); weights fp32 [d] or None
    (ones); eps None: no norm.  rope None: no rotation, else positions int32 [B, L, axes]
    (or [L, axes], shared by the batch).  Returns (q_out, k_out), bf16, None where there was no
    input; an output may be its input (in place)."""
    t = k if q is None else q
    if t is None:
        raise ValueError("qk_norm_rope needs q or k")
    dev = t.get_device()
    B, _, L, d = _shape4("q and k", t)
    H = H_kv = 0
    sq = so = sk = sko = _NO
    qp = qop = kp = kop = None
    if q is not None:
        shape = q.shape
        H = shape[1]
        sq, qp = _rows("q", q, dev, shape)
        q_out = _new(torch.empty_like, q, stream=stream, dev=dev) if q_out is None else q_out
        so, qop = _rows("q_out", q_out, dev, shape)
    if k is not None:
        H_kv = _shape4("k", k)[1]
        shape = (B, H_kv, L, d)
        sk, kp = _rows("k", k, dev, shape)
        k_out = _new(torch.empty_like, k, stream=stream, dev=dev) if k_out is None else k_out
        sko, kop = _rows("k_out", k_out, dev, shape)
    desc = _ROWS.pack(B, H, H_kv, L, d, -1.0 if eps is None else eps, *sq, *sk, *_NO, *so, *sko, *_NO, 0, 0)
    _launch(dev, load().sfa_qk_norm_rope,
            (desc, _rope_desc(rope, positions, layout, dev, B, L), qp, kp, _weight("q_weight", q_weight, dev, d),
             _weight("k_weight", k_weight, dev, d), qop, kop), stream, "sfa_qk_norm_rope")
    return None if q is None else q_out, None if k is None else k_out


def cache_write(cache: FrameCache, k, v, table, start, lens=None, dev_status=None, stream=None):
    """Write new keys and values bf16 [B, H_kv, L, d] into the cache: token i of (b, h) becomes
    logical token start[b][h] + i.  table int32 [B, N] or [B, H_kv, N] of page numbers, start
    int32 [B] or [B, H_kv], lens int32 [B] (rows from there on are padding) or None."""
    dev = k.get_device()
    shape = _shape4("k", k)
    sk, kp = _rows("k", k, dev, shape)
    sv, vp = _rows("v", v, dev, shape)
    B, H_kv, L, d = shape
    cd = _cache_desc(cache, table, dev, B, H_kv, d)
    desc = _ROWS.pack(B, 0, H_kv, L, d, -1.0, *_NO, *sk, *sv, *_NO, *_NO, *_NO, *_per_head("start", start, dev, B, H_kv))
    _launch(dev, load().sfa_cache_write,
            (desc, cd, kp, vp, start.data_ptr(), _lens("lens", lens, dev, B), _status(dev_status, dev)), stream,
            "sfa_cache_write")


def cache_append(cache: FrameCache, q, k, v, table, start, lens=None, rope: RopeTable | None = None, positions=None,
                 q_weight=None, k_weight=None, eps: float | None = 1e-6, layout: str = "interleaved", q_out=None,
                 dev_status=None, stream=None):
    """qk_norm_rope of q and k, and cache_write of those keys and v, in one pass (the bf16 keys
    are not written).  Arguments as theirs; returns q_out.  Padding rows of q_out (from lens[b]
    on) are left as they are."""
    dev = q.get_device()
    shape = _shape4("q", q)
    B, H, L, d = shape
    H_kv = _shape4("k", k)[1]
    kv_shape = (B, H_kv, L, d)
    sq, qp = _rows("q", q, dev, shape)
    sk, kp = _rows("k", k, dev, kv_shape)
    sv, vp = _rows("v", v, dev, kv_shape)
    q_out = _new(torch.empty_like, q, stream=stream, dev=dev) if q_out is None else q_out
    so, qop = _rows("q_out", q_out, dev, shape)
    cd = _cache_desc(cache, table, dev, B, H_kv, d)
    desc = _ROWS.pack(B, H, H_kv, L, d, -1.0 if eps is None else eps, *sq, *sk, *sv, *so, *_NO, *_NO,
                      *_per_head("start", start, dev, B, H_kv))
    _launch(dev, load().sfa_cache_append,
            (desc, _rope_desc(rope, positions, layout, dev, B, L), cd, qp, kp, vp,
             _weight("q_weight", q_weight, dev, d), _weight("k_weight", k_weight, dev, d), qop, start.data_ptr(),
             _lens("lens", lens, dev, B), _status(dev_status, dev)), stream, "sfa_cache_append")
    return q_out


def cache_read(cache: FrameCache, table, start, L: int, lens=None, k_out=None, v_out=None, H_kv: int | None = None,
               dev_status=None, stream=None):
    """Logical tokens start[b][h] + i, i < min(L, lens[b]), of every (b, h) back as bf16
    [B, H_kv, L, d]: (k_out, v_out).  Other rows are left as they are (zero where the outputs
    are allocated here).  H_kv: key heads, where neither the pool nor the table says so."""
    pool, t = _shape4("cache.k", cache.k), table.shape
    dev, B, d = cache.k.get_device(), t[0], pool[3]
    if H_kv is None:
        H_kv = _shape4("k_out", k_out)[1] if k_out is not None else max(pool[1], t[1] if len(t) == 3 else 1)
    shape = (B, H_kv, int(L), d)
    if k_out is None:
        k_out = _new(torch.zeros, shape, dtype=_BF16, device=cache.k.device, stream=stream, dev=dev)
    if v_out is None:
        v_out = _new(torch.zeros, shape, dtype=_BF16, device=cache.k.device, stream=stream, dev=dev)
    sk, kp = _rows("k_out", k_out, dev, shape)
    sv, vp = _rows("v_out", v_out, dev, shape)
    cd = _cache_desc(cache, table, dev, B, H_kv, d)
    desc = _ROWS.pack(B, 0, H_kv, shape[2], d, -1.0, *_NO, *_NO, *_NO, *_NO, *sk, *sv,
                      *_per_head("start", start, dev, B, H_kv))
    _launch(dev, load().sfa_cache_read,
            (desc, cd, start.data_ptr(), _lens("lens", lens, dev, B), kp, vp, _status(dev_status, dev)), stream,
            "sfa_cache_read")
    return k_out, v_out


def _key_heads(cache, table, kv_lens):
    """Key heads as the pool, the table or the lengths have them."""
    n, t = cache.k.shape[1], table.shape
    if n == 1 and len(t) == 3:
        n = t[1]
    if n == 1 and kv_lens.dim() == 2:
        n = kv_lens.shape[1]
    return n


def forward_cache_workspace_bytes(q, cache: FrameCache, table, kv_lens, max_kv: int = 0, H_kv: int | None = None) -> int:
    """Device workspace bytes of forward_cache for these shapes."""
    B, H, Lq, d = _shape4("q", q)
    if H_kv is None:
        H_kv = _key_heads(cache, table, kv_lens)
    cd = _cache_desc(cache, table, q.get_device(), B, H_kv, d)
    desc = _ATTN.pack(B, H, H_kv, Lq, d, 1.0, 0, max_kv, *_NO, *_NO, 0, 0, 0, 0)
    out = ctypes.c_size_t(0)
    _check(load().sfa_forward_cache_workspace(desc, cd, ctypes.byref(out)), "sfa_forward_cache_workspace")
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
    LSE = -inf, so the result merges with other branches by lse_merge.  debug_flags: SFA_DEBUG_*
    test hooks, 0 in normal use."""
    dev = q.get_device()
    shape = _shape4("q", q)
    sq, qp = _rows("q", q, dev, shape)
    out = _new(torch.empty_like, q, stream=stream, dev=dev) if out is None else out
    so, op = _rows("out", out, dev, shape)
    B, H, Lq, d = shape
    if lse is None:
        lse = _new(torch.empty, shape[:3], dtype=_F32, device=q.device, stream=stream, dev=dev)
    elif lse.dtype is not _F32 or lse.get_device() != dev or lse.shape != shape[:3] or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 tensor {tuple(shape[:3])} on device {dev}")
    if H_kv is None:
        H_kv = _key_heads(cache, table, kv_lens)
    cd = _cache_desc(cache, table, dev, B, H_kv, d)
    desc = _ATTN.pack(B, H, H_kv, Lq, d, 1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0, max_kv,
                      *sq, *so, *_per_head("kv_lens", kv_lens, dev, B, H_kv), timeout_us, debug_flags)
    lib = load()
    if workspace is None:
        need = ctypes.c_size_t(0)
        _check(lib.sfa_forward_cache_workspace(desc, cd, ctypes.byref(need)), "sfa_forward_cache_workspace")
        if need.value:
            workspace = _new(torch.empty, need.value, dtype=torch.uint8, device=q.device, stream=stream, dev=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _launch(dev, lib.sfa_forward_cache,
            (desc, cd, qp, kv_lens.data_ptr(), _lens("q_lens", q_lens, dev, B), op, lse.data_ptr(), ws, ws_bytes,
             _status(dev_status, dev)), stream, "sfa_forward_cache")
    return out, lse
