"""A sink whose score stands far above the others', as trained models have: the
many other keys' weights are tiny, and together still make up the output.

P is rounded to the 16-bit format relative to the row's largest weight: bf16 to
half a step of its own size, fp16 the same or 2^-32, half a step of its smallest
numbers when P is 2^7 at the largest.  The bound is that of the rounded P and
out, with fp32 arithmetic inside."""
import math

import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import FP32, HALF, Cache

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
LEAST = {BF16: 0.0, F16: 2.0 ** -32}


def keys(n, Hkv, D, above, dtype):
    """q, k, v such that key 0 scores `above` and the others about 0; v is 0 there and about 1 elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(n)
    k = 0.02 * torch.randn((n, Hkv, D), generator=g, device="cuda")
    v = 1 + 0.1 * torch.randn((n, Hkv, D), generator=g, device="cuda")
    k[0] = above * math.sqrt(D) / D
    v[0] = 0
    return k.to(dtype), v.to(dtype)


def check(out, q, k, v, first, window, sinks, dtype):
    """out, q [n, D] at positions first.., one head's k, v [m, D]."""
    x = first + torch.arange(len(q), device="cuda")[:, None]
    j = torch.arange(len(k), device="cuda")[None]
    see = (j <= x) & ((x - j < window) | (j < sinks) | (window == 0))
    s = (q.double() @ k.double().T / math.sqrt(q.shape[1])).masked_fill(~see, -math.inf)
    p = torch.softmax(s, -1)
    ref, size = p @ v.double(), p @ v.double().abs()
    u = HALF[dtype]
    bound = u * ref.abs() + (u + FP32) * size + LEAST[dtype] * p.amax(-1, keepdim=True) * (see.double() @ v.double().abs())
    off = (out.double() - ref).abs()
    assert bool((off <= bound + 2.0 ** -24).all()), f"worst {float((off / ref.abs().clamp_min(1e-9)).max()):.1e} of out"


@pytest.mark.parametrize("above", [12.0, 15.0, 16.5])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("N,H,Hkv,D,window,sinks", [(4000, 2, 1, 64, 4000, 0), (3000, 2, 2, 128, 1500, 4)])
def test_window(N, H, Hkv, D, window, sinks, dtype, above):
    k, v = keys(N, Hkv, D, above, dtype)
    q = torch.ones((1, N, H, D), dtype=dtype, device="cuda")
    out, _ = bd.window_attn(q, k[None], v[None], window, sinks)
    for h in range(H):
        f = h * Hkv // H
        check(out[0, :, h], q[0, :, h], k[:, f], v[:, f], 0, window, sinks, dtype)


@pytest.mark.parametrize("above", [15.0, 16.5])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nq,n,H,Hkv,D", [(1, 9000, 4, 2, 64), (3, 4000, 2, 1, 128), (40, 9000, 2, 1, 64), (600, 5000, 4, 2, 128)])
def test_paged(nq, n, H, Hkv, D, dtype, above):
    cache = Cache([n], 64, Hkv, D, dtype, 3)
    cache.k[0], cache.v[0] = keys(n, Hkv, D, above, dtype)
    pages = cache.table[0].long()
    for pool, rows in ((cache.k_pages, cache.k[0]), (cache.v_pages, cache.v[0])):
        whole = torch.full((len(pages) * 64, Hkv, D), float("nan"), dtype=dtype, device="cuda")
        whole[:n] = rows
        pool[pages] = whole.view(len(pages), 64, Hkv, D)
    q = torch.ones((nq, H, D), dtype=dtype, device="cuda")
    cu = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
    families = [bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_TCGEN05]
    for impl in families:
        out, _ = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, nq, impl=impl)
        for h in range(H):
            f = h * Hkv // H
            check(out[:, h], q[:, h], cache.k[0][:, f], cache.v[0][:, f], n - nq, 0, 0, dtype)
    assert bd.longnet_last_device_status() == 0
