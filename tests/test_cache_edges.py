"""What the 8-bit frame cache's calls refuse beside wrong shapes and types (CPU)."""
import pytest
import torch

from test_cache_abi import sfa  # noqa: F401


def test_a_negative_eps_is_no_request_for_no_norm(sfa):  # noqa: F811
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    cache = sfa.cache_create(1, 16, 64, device="cpu")
    table, start = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for eps in (-1e-6, -1.0, float("-inf")):
        with pytest.raises(ValueError, match="eps"):
            sfa.qk_norm_rope(q, eps=eps)
        with pytest.raises(ValueError, match="eps"):
            sfa.cache_append(cache, q, q, q, table, start, eps=eps)
    for eps in (None, 0.0, -0.0, 1e-6):  # (refused for what the tensors are)
        with pytest.raises(ValueError, match="CUDA"):
            sfa.qk_norm_rope(q, eps=eps)


def test_rope_tables_without_a_meaning(sfa):  # noqa: F811
    inf, nan = float("inf"), float("nan")
    yarn = dict(scaling="yarn", factor=2.0, original_len=64)
    for kw in (dict(factor=inf, scaling="linear"), dict(factor=nan), dict(theta=inf), dict(theta=nan), dict(yarn, beta_fast=1.0),
               dict(yarn, beta_fast=1.0, beta_slow=32.0), dict(yarn, beta_slow=nan)):
        with pytest.raises(ValueError):
            sfa.rope_table((64,), device="cpu", **kw)


def test_yarn_blends_by_turns(sfa):  # noqa: F811
    """Pair by pair from the paper's formula."""
    import math
    n, L, factor, fast, slow = 64, 4096, 8.0, 32.0, 1.0
    t = sfa.rope_table((n,), scaling="yarn", factor=factor, original_len=L, device="cpu").inv_freq.tolist()
    for i, f in enumerate(t):
        base = 10000.0 ** (-2 * i / n)
        turns = L * base / (2 * math.pi)
        gamma = 0.0 if turns < slow else 1.0 if turns > fast else (turns - slow) / (fast - slow)
        assert math.isclose(f, (1 - gamma) * base / factor + gamma * base, rel_tol=1e-14)


def _views():
    from test_cache_abi import _structs
    rows, cache, rope = _structs()  # contiguous [2, 4, 8, 64] and [2, 2, 8, 64]
    return rows, cache, rope


def test_outputs_at_an_inputs_address(sfa):  # noqa: F811
    """In place means the same rows at the same places; an output is nobody else's memory."""
    import ctypes

    from test_cache_abi import GOOD
    lib, r = sfa.load(), ctypes.byref
    a, b, c, x = (GOOD + (i << 16) for i in range(4))

    def norm(rows, *args):
        return lib.sfa_qk_norm_rope(r(rows), None, *args[:2], None, None, *args[2:], None)

    def append(rows, q, k, v, q_out):
        return lib.sfa_cache_append(r(rows), None, r(cache), q, k, v, None, None, q_out, GOOD, None, None, None)
    for t, args in (("q", (a, None, a, None)), ("k", (None, a, None, a))):
        rows, cache, _ = _views()
        for i, s in enumerate((4 * 8 * 64, 64, 4 * 64)):  # [B, L, heads, d] over the same memory
            setattr(rows, f"{t}_out_stride{i}", s)
        assert norm(rows, *args) == 1
        if t == "q":
            assert append(rows, a, b, c, a) == 1
    rows, cache, _ = _views()
    for args in ((a, b, b, x), (a, b, x, a), (a, b, x, x), (a, a, a, a)):
        assert norm(rows, *args) == 1
    for args in ((a, b, c, b), (a, b, c, c)):
        assert append(rows, *args) == 1
    assert lib.sfa_cache_read(r(rows), r(cache), GOOD, None, a, a, None, None) == 1


def test_attention_output_at_the_queries_address(sfa):  # noqa: F811
    from test_cache_abi import GOOD, _attn, _attn_call, _structs
    _, cache, _ = _structs()
    d = _attn(sfa)  # contiguous [2, 4, 8, 64]
    for i, s in enumerate((4 * 8 * 64, 64, 4 * 64)):
        setattr(d, f"o_stride{i}", s)
    assert _attn_call(sfa, d, cache, q=GOOD, o=GOOD) == 1
