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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("window,sinks", [(100, 0), (130, 5), (513, 129), (64, 128)])
@pytest.mark.parametrize("nq", [1, 3, 70])
def test_pages_behind_the_window_may_be_given_back(nq, window, sinks, page, dtype):
    """Entries of pages with only keys of [128 ceil(sinks / 128), 128 floor((x0 - window + 1) / 128)) are not read."""
    H, Hkv, D, lens = 4, 2, 64, [2000, 1023, 700]
    cache = Cache(lens, page, Hkv, D, dtype, nq)
    g = torch.Generator(device="cuda").manual_seed(nq)
    q = torch.randn((3 * nq, H, D), generator=g, device="cuda").to(dtype)
    cu = torch.tensor([i * nq for i in range(4)], dtype=torch.int32, device="cuda")
    table, k_pages, v_pages, freed = cache.table.clone(), cache.k_pages.clone(), cache.v_pages.clone(), 0
    for s, n in enumerate(lens):
        a, b = -(-sinks // 128) * 128, (n - nq - window + 1) // 128 * 128
        for i in range(-(-a // page), b // page):
            k_pages[table[s, i]] = v_pages[table[s, i]] = float("nan")
            table[s, i] = -1 if i % 2 else 1 << 29
            freed += 1
        if page < 256:  # the keys of a kept page that lie in the range
            for j in range(a, b):
                if 0 <= table[s, j // page] < k_pages.shape[0]:
                    k_pages[table[s, j // page], j % page] = v_pages[table[s, j // page], j % page] = float("nan")
    assert freed
    families = [bd.LONGNET_IMPL_AUTO] if dtype == F32 else [bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_TCGEN05, bd.LONGNET_IMPL_SIMT]
    for impl in families:
        def run(k, v, t):
            w = torch.zeros((3, Hkv, cache.table.shape[1] * page), device="cuda")
            out, lse = bd.paged_attn(q, k, v, cu, cache.kv_len, t, nq, window, sinks, w, impl=impl)
            return out, lse, w

        want, got = run(cache.k_pages, cache.v_pages, cache.table), run(k_pages, v_pages, table)
        assert bd.longnet_last_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, got))
