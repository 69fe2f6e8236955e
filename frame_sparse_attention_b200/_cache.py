"""Binding of the 8-bit frame cache: norm and rotation of new queries and keys, writing and
reading the cache, and attention over it (sfa_qk_norm_rope, sfa_cache_write,
sfa_cache_append, sfa_cache_read, sfa_forward_cache in include/sfa.h).

Like the rest of the binding it only marshals tensors; every call runs on the tensors'
device, on that device's current stream unless one is given.  These calls are a few microseconds
of GPU time at a single token, so their tensors are checked and marshalled in C++ (_bind.so,
csrc/sfa_bind.cpp) instead of through ctypes.
"""
from __future__ import annotations

import importlib
import math
import os
import re
import sys
from typing import NamedTuple

import torch

from ._lib import _PKG, _require, load

CACHE_BLOCK = 32  # elements of a cached row that share a scale
ROPE_MAX_AXES = 4


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
    own row of the page table and can keep other frames than its neighbours).  cache_write and
    cache_append never store the formats' NaNs; in a pool filled otherwise they are read as
    numbers (codes as 480, scales as 2^128)."""
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
    keeps those that turn more than beta_fast times, blends the ones between linearly in their
    number of turns, as the paper has it, and scales rotated values by 0.1 ln(factor) + 1.
    (Many published checkpoints blend linearly in the pair's index instead, between bounds
    rounded to whole indices: a model trained so needs a RopeTable of its own frequencies.)"""
    dims = [int(n) for n in axis_dims]
    _require(0 < len(dims) <= ROPE_MAX_AXES and all(n >= 0 and n % 2 == 0 for n in dims) and sum(dims) > 0,
             "expected 1 to 4 even axis dimensions")
    _require(scaling in ("none", "linear", "ntk", "yarn"), "expected scaling in (none, linear, ntk, yarn)")
    _require(0 < factor < math.inf and 0 < theta < math.inf, "expected finite factor > 0 and theta > 0")
    _require(scaling != "yarn" or original_len > 0, "yarn needs original_len")
    _require(scaling != "yarn" or beta_fast > beta_slow, "yarn needs beta_fast > beta_slow")
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


# ---------------------------------------------------------------- the extension module
_bind = None


def _load_bind():
    global _bind
    load()  # the library that it calls
    path = os.path.join(_PKG, "_bind.so")
    how = "build it with `python -m frame_sparse_attention_b200.build`"
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: {how}")
    try:
        module = importlib.import_module("._bind", __package__)
    except ImportError as e:
        raise RuntimeError(f"{path} does not load ({e}): {how}") from e
    # objects of another PyTorch or interpreter may be laid out otherwise
    torch_version = re.match(r"\d+\.\d+\.\d+", torch.__version__)
    have = f"torch {torch_version.group() if torch_version else torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"
    if module.built_for != have:
        raise RuntimeError(f"{path} was built for {module.built_for}, this is {have}: {how}")
    _bind = module
    return _bind


class _Desc:
    """A descriptor of include/sfa.h, with the size that the extension module compiles it to."""

    def __init__(self, name):
        self.name = name

    @property
    def size(self):
        return getattr(_bind or _load_bind(), "sizeof_" + self.name)


_CACHE, _ROPE, _ROWS, _ATTN = map(_Desc, ("cache", "rope", "rows", "attn"))


def qk_norm_rope(q, k=None, rope: RopeTable | None = None, positions=None, q_weight=None, k_weight=None,
                 eps: float | None = 1e-6, layout: str = "interleaved", q_out=None, k_out=None, stream=None):
    """RMS norm of every head's query and key row and their rotary positions, in one pass.

    q bf16 [B, H, L, d], k bf16 [B, H_kv, L, d] (either may be None); weights fp32 [d] or None
    (ones); eps None: no norm.  rope None: no rotation, else positions int32 [B, L, axes]
    (or [L, axes], shared by the batch).  Returns (q_out, k_out), bf16, None where there was no
    input; an output may be its input (in place, under the same strides) and overlap nothing else."""
    return (_bind or _load_bind()).qk_norm_rope(q, k, rope, positions, q_weight, k_weight, eps, layout, q_out, k_out, stream)


def cache_write(cache: FrameCache, k, v, table, start, lens=None, dev_status=None, stream=None):
    """Write new keys and values bf16 [B, H_kv, L, d] into the cache: token i of (b, h) becomes
    logical token start[b][h] + i.  table int32 [B, N] or [B, H_kv, N] of page numbers, start
    int32 [B] or [B, H_kv], lens int32 [B] (rows from there on are padding) or None."""
    (_bind or _load_bind()).cache_write(cache, k, v, table, start, lens, dev_status, stream)


def cache_append(cache: FrameCache, q, k, v, table, start, lens=None, rope: RopeTable | None = None, positions=None,
                 q_weight=None, k_weight=None, eps: float | None = 1e-6, layout: str = "interleaved", q_out=None,
                 dev_status=None, stream=None):
    """qk_norm_rope of q and k, and cache_write of those keys and v, in one pass (the bf16 keys
    are not written).  Arguments as theirs; returns q_out.  Padding rows of q_out (from lens[b]
    on) are left as they are (zero where it is allocated here)."""
    return (_bind or _load_bind()).cache_append(cache, q, k, v, table, start, lens, rope, positions, q_weight, k_weight, eps,
                                                layout, q_out, dev_status, stream)


def cache_read(cache: FrameCache, table, start, L: int, lens=None, k_out=None, v_out=None, H_kv: int | None = None,
               dev_status=None, stream=None):
    """Logical tokens start[b][h] + i, i < min(L, lens[b]), of every (b, h) back as bf16
    [B, H_kv, L, d]: (k_out, v_out).  Other rows are left as they are (zero where the outputs
    are allocated here).  H_kv: key heads, where neither the pool nor the table says so."""
    return (_bind or _load_bind()).cache_read(cache, table, start, L, lens, k_out, v_out, H_kv, dev_status, stream)


def forward_cache_workspace_bytes(q, cache: FrameCache, table, kv_lens, max_kv: int = 0, H_kv: int | None = None) -> int:
    """Device workspace bytes of forward_cache for these shapes (kv_lens as in the call: one length for
    all heads or one each)."""
    return (_bind or _load_bind()).forward_cache_workspace(q, cache, table, kv_lens, max_kv, H_kv)


def forward_cache(q, cache: FrameCache, table, kv_lens, causal: bool = False, q_lens=None, max_kv: int = 0,
                  scale: float | None = None, out=None, lse=None, workspace=None, H_kv: int | None = None,
                  dev_status=None, stream=None, timeout_us: int = 0, debug_flags: int = 0):
    """Attention of new tokens over the cache: (O bf16 like q, LSE fp32 [B, H, Lq]).

    q bf16 [B, H, Lq, d]; kv_lens int32 [B] or [B, H_kv]: logical tokens [0, n) are the keys and
    values.  q_lens int32 [B]: rows from there on are padding, left as they are (O = 0 and LSE = -inf
    where the outputs are allocated here).  causal: the
    rows are the last of the n tokens and see none behind themselves.  max_kv: an upper bound of
    kv_lens, for the split of the work (0: all that the table can hold).  workspace: a uint8
    tensor of forward_cache_workspace_bytes (allocated here when not given).  H_kv: key heads,
    where neither the pool, the table nor kv_lens says so.  Rows that see no key give O = 0,
    LSE = -inf, so the result merges with other branches by lse_merge.  out may be q (in place,
    under the same strides).  debug_flags: SFA_DEBUG_*
    test hooks, 0 in normal use."""
    return (_bind or _load_bind()).forward_cache(q, cache, table, kv_lens, causal, q_lens, max_kv, scale, out, lse, workspace,
                                                 H_kv, dev_status, stream, timeout_us, debug_flags)
