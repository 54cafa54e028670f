"""The paged cache: append, attention of chunks and single tokens, weight sums
and eviction, against their 64-bit forms."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import Cache, evict_reference, paged_reference, within

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
AUTO, SIMT = bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_SIMT

# (new tokens, cached keys) of each sequence; H, Hkv, D, page, window, sinks
CASES = {
    "one token, one key": ([(1, 1)], 1, 1, 16, 8, 0, 0),
    "single tokens": ([(1, 100), (1, 64), (1, 65), (0, 30), (1, 1), (0, 0), (1, 333)], 8, 2, 64, 16, 0, 0),
    "single tokens, long": ([(1, 5000), (1, 2049), (1, 4096)], 4, 4, 128, 64, 0, 0),
    "single tokens, one wide group": ([(1, 700), (1, 31)], 16, 1, 128, 32, 0, 0),
    "single tokens, odd group, window": ([(1, 900), (1, 20)], 6, 2, 32, 16, 128, 4),
    "single tokens, window of one": ([(1, 300)], 2, 1, 64, 256, 1, 0),
    "few tokens": ([(4, 400), (2, 2), (3, 129), (1, 1000)], 8, 2, 64, 16, 0, 0),
    "drafts of 5, window": ([(5, 800), (5, 5), (0, 12)], 12, 4, 128, 64, 200, 66),
    "chunk from nothing": ([(200, 200)], 4, 2, 64, 16, 0, 0),
    "chunks": ([(130, 700), (1, 300), (64, 64), (0, 0), (257, 1500)], 4, 2, 64, 32, 0, 0),
    "chunks, wide heads, window": ([(300, 900), (33, 400)], 6, 2, 128, 128, 150, 4),
    "chunks, narrow heads": ([(100, 513), (300, 301)], 2, 2, 16, 8, 0, 0),
    "chunks, group of 7, sinks past a block": ([(90, 1100)], 7, 1, 32, 16, 64, 140),
    "long chunk over a long cache": ([(140, 6000)], 2, 1, 64, 256, 0, 0),
    "more tokens than keys": ([(5, 3), (40, 8)], 2, 1, 64, 16, 0, 0),
    "no new tokens": ([(0, 100), (0, 0)], 4, 2, 64, 16, 0, 0),
    "wider groups than a tile": ([(2, 300), (1, 20)], 130, 1, 32, 16, 0, 0),
    "group of a whole tile": ([(3, 200), (1, 90)], 128, 1, 64, 32, 50, 2),
    "many short sequences": ([(1 + i % 3, 3 + i % 40) for i in range(330)], 20, 1, 16, 8, 0, 0),
    "very many sequences": ([(1, 1 + i % 17) for i in range(2100)], 1, 1, 16, 8, 0, 0),
    "window, long cache, few tokens": ([(6, 9000), (2, 4000)], 8, 1, 128, 64, 3000, 5),
}


def setup(case, dtype, seed=3, pad=3):
    seqs, H, Hkv, D, page, window, sinks = CASES[case]
    nq, lens = [n for n, _ in seqs], [m for _, m in seqs]
    cache = Cache(lens, page, Hkv, D, dtype, seed, wide=max(-(-m // page) for m in lens) + 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(nq) + pad
    q = torch.randn((T, H, D), generator=g, device="cuda").to(dtype)
    cu = torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32, device="cuda")
    return cache, q, nq, cu, window, sinks


def attend(cache, q, cu, max_q, window, sinks, impl, weights=None):
    T, H, D = q.shape
    out = torch.full((T, H, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    n = bd.longnet_paged_workspace_bytes(cu.numel() - 1, max_q, H, cache.Hkv, D, cache.page, cache.table.shape[1],
                                         window, sinks, q.dtype, weights is not None)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, max_q, window, sinks, weights, out,
                  lse, ws[:n], impl)
    assert bool((ws[n:] == 255).all()), "write past the workspace"
    return out, lse


def families(dtype):
    return [AUTO] if dtype == F32 else [AUTO, SIMT, bd.LONGNET_IMPL_TCGEN05, bd.LONGNET_IMPL_DECODE]


def refused(impl, case, dtype, more=0):
    """The few-token family takes at most 16 query rows per key/value head."""
    seqs, H, Hkv = CASES[case][:3]
    if impl == bd.LONGNET_IMPL_TCGEN05:
        return H // Hkv > 128
    return impl == bd.LONGNET_IMPL_DECODE and ((max(1, *(n for n, _ in seqs)) + more) * (H // Hkv) > 16
                                               or len(seqs) > 2048)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("case", CASES)
def test_attention_and_weights(case, dtype):
    cache, q, nq, cu, window, sinks = setup(case, dtype)
    out, lse, w, b_out = paged_reference(cache, q, nq, window, sinks)
    n = sum(nq)
    top = max(1, *nq)
    for impl in families(dtype):
        if refused(impl, case, dtype):
            continue
        for max_q in (top, top + 3):
            if refused(impl, case, dtype, max_q - top):
                with pytest.raises(bd.LongNetError):
                    attend(cache, q, cu, max_q, window, sinks, impl)
                continue
            got, got_lse = attend(cache, q, cu, max_q, window, sinks, impl)
            assert bd.longnet_last_device_status() == 0
            within(f"out {impl}", got[:n], out[:n], b_out[:n])
            within(f"lse {impl}", got_lse[:n], lse[:n], torch.full_like(lse[:n], 1e-4))
            assert bool((got[n:] == 7).all()) and bool((got_lse[n:] == 7).all()), "rows of no sequence were written"
        start = torch.rand(w.shape, device="cuda")
        weights = start.clone()
        again, again_lse = attend(cache, q, cu, top, window, sinks, impl, weights)
        assert bd.longnet_last_device_status() == 0
        within(f"out with weights {impl}", again[:n], out[:n], b_out[:n])
        # a weight is a sum of e^{s - lse} in fp32
        within(f"weights {impl}", weights, start.double() + w, 1e-4 * w + 1e-6)
        twice = start.clone()
        attend(cache, q, cu, top, window, sinks, impl, twice)
        assert torch.equal(weights, twice), "the same inputs gave other bits"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [8, 64])
def test_append(dtype, page):
    Hkv, D = 3, 32
    lens, nq = [20, 0, 65, 7], [5, 0, 65, 1]
    cache = Cache(lens, page, Hkv, D, dtype, 5, wide=12)
    T = sum(nq) + 2
    k_tok, v_tok = (torch.randn((T, Hkv, D), device="cuda").to(dtype) for _ in range(2))
    cu = torch.tensor([0, 5, 5, 70, 71], dtype=torch.int32, device="cuda")
    k, v = cache.k_pages.clone(), cache.v_pages.clone()
    weights = torch.ones((4, Hkv, 12 * page), device="cuda")
    want_w = weights.clone()
    bd.paged_append(k_tok, v_tok, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, weights)
    assert bd.longnet_last_device_status() == 0
    for s in range(4):
        for i in range(nq[s]):
            x = lens[s] - nq[s] + i
            at = int(cache.table[s, x // page])
            k[at, x % page], v[at, x % page] = k_tok[int(cu[s]) + i], v_tok[int(cu[s]) + i]
            want_w[s, :, x] = 0
    eq = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731  (NaN slots too)
    assert eq(cache.k_pages, k) and eq(cache.v_pages, v) and torch.equal(weights, want_w)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D,page,budget,sinks,recent", [
    (64, 16, 40, 4, 8), (16, 8, 1, 0, 0), (32, 64, 64, 0, 64), (128, 32, 100, 100, 0), (64, 256, 300, 2, 0),
    (128, 16, 7, 3, 4)])
def test_evict(dtype, D, page, budget, sinks, recent):
    Hkv, lens = 3, [0, 1, budget, budget + 1, 333, 5000]
    wide = -(-5000 // page)
    cache = Cache(lens, page, Hkv, D, dtype, 7, wide=wide)
    g = torch.Generator().manual_seed(1)
    w = torch.exp(2 * torch.randn((6, Hkv, wide * page), generator=g))
    w[:, :, ::3] = 0.0  # many ties
    w[3, 0, :50] = 1.5
    w[4, 1, 5:300:7] = float("nan")
    w[4, 2, 9] = float("inf")
    w[5, 0, 3:4000] = -0.0
    w[5, 1, 100:105] = float("-inf")
    weights = w.cuda()
    out_wide = -(-budget // page) + 1
    n_out = 6 * out_wide + 2
    new_table = torch.randperm(n_out, generator=g)[:6 * out_wide].view(6, out_wide).int().cuda()
    k_out = torch.full((n_out, page, Hkv, D), 3.0, dtype=dtype, device="cuda")
    v_out = torch.full_like(k_out, 3.0)
    kept, new_len, new_w = bd.cache_evict(cache.k_pages, cache.v_pages, weights, cache.kv_len, cache.table, k_out,
                                          v_out, new_table, budget, sinks, recent)
    assert bd.longnet_last_device_status() == 0
    want = evict_reference(w, lens, budget, sinks, recent)
    assert torch.equal(kept.cpu().long(), want)
    assert new_len.tolist() == [min(n, budget) for n in lens]
    k_want, v_want = torch.full_like(k_out, 3.0), torch.full_like(v_out, 3.0)
    w_want = torch.zeros_like(new_w)
    for s, n in enumerate(lens):
        m = min(n, budget)
        for f in range(Hkv):
            sel = want[s, f, :m].cuda()
            j = torch.arange(m, device="cuda")
            w_want[s, f, :m] = weights[s, f, sel]
            pg = new_table[s].long()[j // page]
            k_want[pg, j % page, f] = cache.k[s][sel, f]
            v_want[pg, j % page, f] = cache.v[s][sel, f]
    assert torch.equal(k_out, k_want) and torch.equal(v_out, v_want)
    assert torch.equal(new_w.view(torch.int32), w_want.view(torch.int32))


def test_prompt_then_tokens_then_eviction():
    """A program's run: a prompt in chunks, single tokens with their weights
    gathered, an eviction into free pages of the same pool, more tokens."""
    H, Hkv, D, page, dtype = 8, 2, 64, 16, BF16
    cache = Cache([0, 0], page, Hkv, D, dtype, 2, spare=64, wide=20)
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    weights = torch.full((2, Hkv, 20 * page), 9.0, device="cuda")
    table = cache.table.cpu()
    for s in range(2):
        for i in range(20):
            table[s, i] = cache.free.pop()
    cache.table.copy_(table)
    total_w = torch.zeros_like(weights, dtype=torch.float64)

    def step(nq):
        n = sum(nq)
        k, v, q = rnd(n, Hkv, D), rnd(n, Hkv, D), rnd(n, H, D)
        cu = torch.tensor([0, nq[0], n], dtype=torch.int32, device="cuda")
        at = 0
        for s in range(2):
            cache.k[s] = torch.cat([cache.k[s], k[at:at + nq[s]]])
            cache.v[s] = torch.cat([cache.v[s], v[at:at + nq[s]]])
            cache.lens[s] += nq[s]
            at += nq[s]
        cache.kv_len.copy_(torch.tensor(cache.lens, dtype=torch.int32))
        bd.paged_append(k, v, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, weights)
        out, lse = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, max(nq),
                                 weights=weights)
        ref, rlse, w, b = paged_reference(cache, q, nq, 0, 0)
        within("out", out, ref, b)
        return w

    for nq in ((100, 37), (60, 1), (1, 1), (1, 1), (0, 3)):
        total_w += step(nq)
    for s in range(2):
        n = cache.lens[s]
        within("weights", weights[s, :, :n], total_w[s, :, :n], 1e-4 * total_w[s, :, :n] + 1e-5)
    wide = 20
    new_table = torch.tensor([[cache.free.pop() if i < 5 else -1 for i in range(wide)] for _ in range(2)],
                             dtype=torch.int32, device="cuda")
    kept, new_len, new_w = bd.cache_evict(cache.k_pages, cache.v_pages, weights, cache.kv_len, cache.table,
                                          cache.k_pages, cache.v_pages, new_table, 64, 4, 16)
    for s in range(2):
        m = int(new_len[s])
        sel = kept[s, :, :m].long()
        for name in ("k", "v"):
            old = getattr(cache, name)[s]
            getattr(cache, name)[s] = torch.stack([old[sel[f], f] for f in range(Hkv)], 1)
        cache.lens[s] = m
    weights = new_w
    cache.table.copy_(new_table)
    cache.kv_len.copy_(new_len)
    total_w = new_w.double()
    for nq in ((1, 1), (1, 0), (10, 3)):
        total_w += step(nq)
    assert bd.longnet_last_device_status() == 0
    for s in range(2):
        n = cache.lens[s]
        within("weights", weights[s, :, :n], total_w[s, :, :n], 1e-4 * total_w[s, :, :n] + 1e-5)


def test_served_rows_equal_trained_rows():
    """The window mask of training and of serving is one: a prompt served in
    chunks gives the rows of the full-sequence forward."""
    N, H, Hkv, D, page = 500, 4, 2, 64, 32
    cache = Cache([N], page, Hkv, D, BF16, 6)
    q = torch.randn((N, H, D), device="cuda").to(BF16)
    out, lse = bd.window_attn(q[None], cache.k[0][None].contiguous(), cache.v[0][None].contiguous(), 70, 5)
    for a, b in ((0, 200), (200, 201), (201, 500)):
        cache.kv_len.fill_(b)
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        o, l = bd.paged_attn(q[a:b].contiguous(), cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, b - a,
                             70, 5)
        u = torch.finfo(BF16).eps / 2
        # each side within u |out| + u sum P |v| of the exact row; |v| < 5 here
        assert float((o.float() - out[0, a:b].float()).abs().max()) <= 2 * u * (5 + 5)
        assert float((l - lse[0, :, a:b].T).abs().max()) <= 2e-4


def test_captured_step_serves_changing_batches():
    """One captured append + attend, replayed with other lengths, tables and tokens."""
    H, Hkv, D, page, S, wide = 4, 2, 64, 16, 3, 12
    a = Cache([150, 20, 33], page, Hkv, D, F16, 1, wide=wide)
    T, max_q = 9, 4
    q = torch.zeros((T, H, D), dtype=F16, device="cuda")
    kt, vt = torch.zeros((T, Hkv, D), dtype=F16, device="cuda"), torch.zeros((T, Hkv, D), dtype=F16, device="cuda")
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    pool_k, pool_v = torch.zeros((64, page, Hkv, D), dtype=F16, device="cuda"), None
    pool_v = torch.zeros_like(pool_k)
    kv_len, table = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros((S, wide), dtype=torch.int32, device="cuda")
    weights = torch.zeros((S, Hkv, wide * page), device="cuda")
    out = torch.zeros_like(q)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bd.paged_append(kt, vt, pool_k, pool_v, cu, kv_len, table, weights)
            bd.paged_attn(q, pool_k, pool_v, cu, kv_len, table, max_q, weights=weights, out=out)
        graphs.append(g)
    for r, (lens, nq) in enumerate([([150, 20, 33], [1, 1, 1]), ([4, 0, 180], [4, 0, 2]), ([77, 190, 1], [0, 4, 1])]):
        c = Cache(lens, page, Hkv, D, F16, 10 + r, wide=wide)
        pool_k[:c.k_pages.shape[0]].copy_(c.k_pages)
        pool_v[:c.v_pages.shape[0]].copy_(c.v_pages)
        table.copy_(c.table)
        kv_len.copy_(c.kv_len)
        cu.copy_(torch.tensor([sum(nq[:i]) for i in range(4)], dtype=torch.int32))
        q.normal_()
        at = 0
        for s in range(3):  # the new tokens' rows are those the cache already holds
            kt[at:at + nq[s]] = c.k[s][lens[s] - nq[s]:]
            vt[at:at + nq[s]] = c.v[s][lens[s] - nq[s]:]
            at += nq[s]
        weights.zero_()
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        ref, _, w, b = paged_reference(c, q, nq, 0, 0)
        within("out", out[:at], ref[:at], b[:at])
        within("weights", weights, w, 1e-4 * w + 1e-6)
    assert bd.longnet_last_device_status() == 0


def test_bad_lengths_and_pages_are_recorded_and_skipped():
    """Out of range entries are caught by the kernels' own checks: nothing is
    read through them, the status word says so, the other sequence is right."""
    for impl in families(BF16):
        cache, q, nq, cu, _, _ = setup("few tokens", BF16)
        out, lse, _, b = paged_reference(cache, q, nq, 0, 0)
        for what in ("page", "long", "negative"):
            kv_len, table = cache.kv_len.clone(), cache.table.clone()
            if what == "page":
                table[0, 3] = cache.k_pages.shape[0]
            elif what == "long":
                kv_len[0] = table.shape[1] * cache.page + 1
            else:
                kv_len[0] = -1
            got, _ = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, kv_len, table, 4, impl=impl)
            assert bd.longnet_last_device_status() == bd.LONGNET_ERR_DEVICE_BOUNDS, (impl, what)
            within("the other sequences", got[4:10], out[4:10], b[4:10])
        got, _ = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, 3, impl=impl)
        assert bd.longnet_last_device_status() == bd.LONGNET_ERR_DEVICE_BOUNDS  # sequence 0 has 4 tokens
        within("the other sequences", got[4:10], out[4:10], b[4:10])


def test_no_tokens_at_all():
    cache = Cache([5], 8, 1, 16, BF16, 1)
    q = torch.empty((0, 2, 16), dtype=BF16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = bd.paged_attn(q, cache.k_pages, cache.v_pages, cu, cache.kv_len, cache.table, 1)
    assert out.shape == (0, 2, 16) and lse.shape == (0, 2)
    bd.paged_append(q[:, :1].contiguous(), q[:, :1].contiguous(), cache.k_pages, cache.v_pages, cu, cache.kv_len,
                    cache.table)
    assert bd.longnet_last_device_status() == 0


def test_pages_past_two_to_the_31_elements():
    """The last pages of a pool whose offsets do not fit 32 bits."""
    Hkv, D, page, H = 8, 128, 256, 16
    n_pages = 2 ** 31 // (Hkv * D * page) + 12
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    lens, nq = [700, 300], [3, 1]
    cache = Cache(lens, page, Hkv, D, BF16, 11, wide=4)
    k_pages = torch.empty((n_pages, page, Hkv, D), dtype=BF16, device="cuda")
    v_pages = torch.empty_like(k_pages)
    small = cache.k_pages.shape[0]
    k_pages[-small:], v_pages[-small:] = cache.k_pages, cache.v_pages
    table = torch.where(cache.table >= 0, cache.table + (n_pages - small), cache.table)
    q = torch.randn((4, H, D), device="cuda").to(BF16)
    cu = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    out, lse, w, b = paged_reference(cache, q, nq, 0, 0)
    k_tok = torch.cat([cache.k[0][-3:], cache.k[1][-1:]]).contiguous()
    v_tok = torch.cat([cache.v[0][-3:], cache.v[1][-1:]]).contiguous()
    for s in range(2):  # what the append has to bring back
        for x in range(lens[s] - nq[s], lens[s]):
            k_pages[int(table[s, x // page]), x % page] = 0
    bd.paged_append(k_tok, v_tok, k_pages, v_pages, cu, cache.kv_len, table)
    for impl in families(BF16):
        weights = torch.zeros_like(w, dtype=torch.float32)
        got, _ = bd.paged_attn(q, k_pages, v_pages, cu, cache.kv_len, table, 3, weights=weights, impl=impl)
        within(f"out {impl}", got, out, b)
        within(f"weights {impl}", weights, w, 1e-4 * w + 1e-6)
    new_table = n_pages - small - torch.tensor([[1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    kept, new_len, _ = bd.cache_evict(k_pages, v_pages, w.float(), cache.kv_len, table, k_pages, v_pages, new_table, 400, 4,
                                      50)
    assert bd.longnet_last_device_status() == 0 and new_len.tolist() == [400, 300]
    for s in range(2):
        n = int(new_len[s])
        j = torch.arange(n, device="cuda")
        for f in (0, Hkv - 1):
            got = k_pages[new_table[s].long()[j // page], j % page, f]
            assert torch.equal(got, cache.k[s][kept[s, f, :n].long(), f])


def test_two_calls_at_once():
    """Two streams, each with its own workspace, give what one after the other gives."""
    cache, q, nq, cu, _, _ = setup("chunks", BF16)
    d_cache, d_q, d_nq, d_cu, _, _ = setup("single tokens, long", BF16)
    want = attend(cache, q, cu, 257, 0, 0, AUTO)
    d_want = attend(d_cache, d_q, d_cu, 1, 0, 0, AUTO)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            a = attend(cache, q, cu, 257, 0, 0, AUTO)
        with torch.cuda.stream(streams[1]):
            b = attend(d_cache, d_q, d_cu, 1, 0, 0, AUTO)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0], want[0]) and torch.equal(b[0], d_want[0])
