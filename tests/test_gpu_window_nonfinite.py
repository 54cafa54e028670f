"""NaN in the sliding-window and paged attention: what a NaN reaches by the
formula is NaN (out, lse and the weights of the keys its row sees), and
everything else has the bits it has without it."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import Cache, visible

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def same(a, b, bad):
    """NaN where bad, the same bits elsewhere."""
    assert bool(a[bad].isnan().all()) and not bool(a[~bad].isnan().any())
    assert torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("impl", [bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_SIMT])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,H,Hkv,D,window,sinks", [(70, 2, 1, 64, 20, 2), (400, 4, 2, 128, 150, 3), (900, 6, 2, 32, 900, 0)])
def test_window(N, H, Hkv, D, window, sinks, dtype, impl):
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k, v = (torch.randn((1, N, h, D), generator=g, device="cuda").to(dtype) for h in (H, Hkv, Hkv))
    out, lse = bd.window_attn(q, k, v, window, sinks, impl)
    # a query row
    q2 = q.clone()
    q2[0, N // 2, 1, 5] = NAN
    bad = torch.zeros((1, N, H), dtype=torch.bool, device="cuda")
    bad[0, N // 2, 1] = True
    out2, lse2 = bd.window_attn(q2, k, v, window, sinks, impl)
    same(out2, out, bad[..., None].expand_as(out))
    same(lse2, lse, bad.transpose(1, 2))
    # a key: every row of its heads that sees it, and no other
    j, f, G = N // 3, Hkv - 1, H // Hkv
    k2 = k.clone()
    k2[0, j, f, 0] = NAN
    bad.zero_()
    bad[0, :, f * G:(f + 1) * G] = visible(torch.arange(N, device="cuda"), torch.tensor(j, device="cuda"), window,
                                           sinks)[:, None]
    out2, lse2 = bd.window_attn(q, k2, v, window, sinks, impl)
    same(out2, out, bad[..., None].expand_as(out))
    same(lse2, lse, bad.transpose(1, 2))
    assert bd.longnet_last_device_status() == 0


# new tokens and cached keys of each sequence, H, Hkv, D, window, sinks: pairs of one CTA and cut ones, row tiles
# whole, cut and alternating, clusters
CASES = [
    ([(1, 90), (1, 300), (1, 2)], 4, 2, 64, 0, 0),
    ([(1, 9000), (1, 3000)], 8, 2, 128, 0, 0),
    ([(4, 700), (2, 2)], 8, 2, 32, 100, 3),
    ([(60, 900), (20, 400)], 4, 2, 64, 0, 0),
    ([(300, 3000), (5, 40)], 4, 2, 64, 200, 70),
    ([(40, 40)] * 330, 2, 1, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("case", CASES, ids=[str(c)[:60] for c in CASES])
def test_paged(case, dtype):
    seqs, H, Hkv, D, window, sinks = case
    nq, lens = [n for n, _ in seqs], [m for _, m in seqs]
    cache = Cache(lens, 16, Hkv, D, dtype, 11)
    G = H // Hkv
    cu = torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((sum(nq), H, D), generator=gen, device="cuda").to(dtype)
    bad_q = q.clone()
    t = nq[0] - 1  # the first sequence's last token
    h = H - 1
    bad_q[t, h, 1] = NAN
    start = torch.rand((len(nq), Hkv, cache.table.shape[1] * 16), device="cuda")
    families = [bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_SIMT]
    if dtype != F32:
        families.append(bd.LONGNET_IMPL_TCGEN05)
        if max(nq) * G <= 16:
            families.append(bd.LONGNET_IMPL_DECODE)
    for impl in families:
        def run(q):
            w = start.clone()
            out, lse = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, max(nq), window,
                                     sinks, w, impl=impl)
            plain, plain_lse = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, max(nq),
                                             window, sinks, impl=impl)
            eq = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
            assert eq(out, plain) and eq(lse, plain_lse)
            return out, lse, w

        (out, lse, w), (out2, lse2, w2) = run(q), run(bad_q)
        assert bd.longnet_last_device_status() == 0
        bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
        bad[t, h] = True
        same(lse2, lse, bad)
        same(out2, out, bad[..., None].expand_as(out))
        bad_w = torch.zeros(w.shape, dtype=torch.bool, device="cuda")
        x = torch.tensor(lens[0] - 1, device="cuda")
        bad_w[0, h // G, :lens[0]] = visible(x, torch.arange(lens[0], device="cuda"), window, sinks)
        same(w2, w, bad_w)
