"""Few-token weights over tables of great capacity: the call runs as several
launches of a few sequences each, whose scores share one bounded workspace."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import Cache, paged_reference, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600000, 100)])
def test_groups_of_sequences(dtype, window, sinks):
    lens, nq, H, Hkv, D, page, wide = [3000, 1, 0, 700, 129], [2, 1, 0, 2, 1], 16, 2, 32, 256, 4096
    # 2 heads of 16 rows and 1M keys are 128 MiB of scores a sequence: groups of 2, 2 and 1
    n = bd.longnet_paged_workspace_bytes(5, 2, H, Hkv, D, page, wide, window, sinks, dtype, True)
    assert n <= (300 << 20)
    cache = Cache(lens, page, Hkv, D, dtype, 3, wide=wide)
    g = torch.Generator(device="cuda").manual_seed(2)
    T = sum(nq)
    q = torch.randn((T + 2, H, D), generator=g, device="cuda").to(dtype)
    cu = torch.tensor([sum(nq[:i]) for i in range(6)], dtype=torch.int32, device="cuda")
    ref, ref_lse, w, b_out = paged_reference(cache, q, nq, window, sinks)
    start = torch.rand(w.shape, device="cuda")
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")

    def run(table):
        weights, out = start.clone(), torch.full_like(q, 7.0)
        _, lse = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, table, 2, window, sinks, weights,
                               out=out, workspace=ws[:n])
        return out, lse, weights

    out, lse, weights = run(cache.table)
    assert bd.longnet_last_device_status() == 0
    assert bool((ws[n:] == 255).all()) and bool((out[T:] == 7).all())
    within("out", out[:T], ref[:T], b_out[:T])
    within("lse", lse[:T], ref_lse[:T], torch.full_like(ref_lse[:T], 1e-4))
    within("weights", weights, start.double() + w, 1e-4 * w + 1e-6)
    again = run(cache.table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(cache.table)
    ws.fill_(255)
    graph.replay()
    for a, b, c in zip((out[:T], lse[:T], weights), (again[0][:T], again[1][:T], again[2]),
                       (captured[0][:T], captured[1][:T], captured[2])):
        assert torch.equal(a, b) and torch.equal(a, c)
    # a page out of range in a later group is recorded, and the other sequences are not affected
    table = cache.table.clone()
    table[3, 0] = cache.k_pages.shape[0]
    other, other_lse, other_w = run(table)
    assert bd.longnet_last_device_status() == bd.LONGNET_ERR_DEVICE_BOUNDS
    keep = [0, 1, 2, 5]
    assert torch.equal(other[keep], out[keep]) and torch.equal(other_lse[keep], lse[keep])
    assert torch.equal(other_w[[0, 1, 2, 4]], weights[[0, 1, 2, 4]])
