"""Calls at the edges of what the paged entry points document."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import Cache

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_batch_without_tokens(dtype):
    cache = Cache([20, 0, 7], 16, 2, 32, dtype, 1)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    weights = torch.rand((3, 2, cache.table.shape[1] * 16), device="cuda")
    before = weights.clone()
    none = torch.empty((0, 2, 32), dtype=dtype, device="cuda")
    bd.paged_append(none, none, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, weights)
    for w in (None, weights):
        out, lse = bd.paged_attn(torch.empty((0, 4, 32), dtype=dtype, device="cuda"), cache.k_pages, cache.v_pages, cu,
                                 cache.kv_len, cache.table, 1, weights=w)
        assert out.shape == (0, 4, 32) and lse.shape == (0, 4)
    assert torch.equal(weights, before) and bd.longnet_last_device_status() == 0
