"""Inputs and references of the 8-bit frame cache tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache as C


def f64(t):
    return t.detach().double().cpu().numpy()


def random_pool(g, sfa, n_pages, heads, page_len, d, device="cuda"):
    """A pool of written rows with uneven scales (FrameCache), every code finite."""
    def half():
        x = torch.from_numpy(g.standard_normal((n_pages, heads, page_len, d)) *
                             np.exp(g.standard_normal((n_pages, heads, page_len, 1))))
        codes, e = C.quantise(x.numpy())
        return (torch.from_numpy(codes).to(torch.float8_e4m3fn).to(device),
                torch.from_numpy(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu).to(device))
    k, ks = half()
    v, vs = half()
    return sfa.FrameCache(k, ks, v, vs)


def empty_pool(sfa, n_pages, heads, page_len, d, device="cuda"):
    """A pool whose unwritten rows hold NaN codes and the largest scale byte."""
    c = sfa.cache_create(n_pages, page_len, d, heads, device)
    for t in c:
        t.view(torch.uint8).fill_(0x7f if t.dtype == torch.float8_e4m3fn else 0xfe)
    return c


def pool_values(cache):
    """(code values, exponents) of keys and values in float64 / int64, NaN codes kept."""
    return [(f64(c), s.view(torch.uint8).cpu().numpy().astype(np.int64) - 127)
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def tables(g, B, rows, n, n_pages):
    """int32 [B][rows][n] of distinct shuffled pages."""
    return g.permutation(n_pages)[: B * rows * n].reshape(B, rows, n).astype(np.int32)


def gather(cache, table, b, h, n):
    """float64 keys and values [n, d] of logical tokens 0 .. n-1 of (b, h)."""
    page_len, heads = cache.k.shape[2], cache.k.shape[1]
    out = []
    for codes, e in pool_values(cache):
        rows = [C.place(table, heads, page_len, b, h, j) for j in range(n)]
        if not rows:
            out.append(np.zeros((0, codes.shape[-1])))
            continue
        at = tuple(np.array(x) for x in zip(*rows))
        out.append(C.dequantise(codes[at], e[at]))
    return out


def strided(t, kind):
    """The same bf16 values with another memory layout: contiguous, [B, L, heads, d], or a slice
    of a wider tensor."""
    if kind == "blhd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "slice":
        wide = torch.full(t.shape[:2] + (t.shape[2] + 3, t.shape[3] + 8), 7.0, dtype=t.dtype, device=t.device)
        view = wide[:, :, 2:-1, 8:]
        view.copy_(t)
        return view
    return t.contiguous()
