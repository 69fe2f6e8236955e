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
