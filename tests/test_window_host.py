"""Argument checks of the sliding-window and paged-cache entry points: refused
on the host, before any device is touched (CPU only)."""
import ctypes

import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd

P = ctypes.c_void_p(0x1000)  # never dereferenced on the host
INVALID, UNSUPPORTED, MISALIGNED = bd.LONGNET_ERR_INVALID_ARG, bd.LONGNET_ERR_UNSUPPORTED, bd.LONGNET_ERR_MISALIGNED


def window(B=1, N=64, H=4, Hkv=2, D=64, window=8, sinks=2, dtype=1, impl=0, ws=1 << 30, **ptrs):
    lib = bd.load_library()
    p = dict(q=P, k=P, v=P, out=P, lse=P)
    p.update({n: ctypes.c_void_p(x) for n, x in ptrs.items() if n in p})
    fwd = lib.longnet_window_attn_fwd(p["q"], p["k"], p["v"], p["out"], p["lse"], B, N, H, Hkv, D, window, sinks, dtype,
                                      impl, None)
    g = {n: ctypes.c_void_p(ptrs[n]) if n in ptrs else P for n in ("dout", "dq", "dk", "dv", "workspace")}
    bwd = lib.longnet_window_attn_bwd(p["q"], p["k"], p["v"], p["out"], p["lse"], g["dout"], g["dq"], g["dk"], g["dv"],
                                      B, N, H, Hkv, D, window, sinks, dtype, impl, g["workspace"], ws, None)
    size = lib.longnet_window_bwd_workspace_bytes(B, N, H, Hkv, D, window, sinks, dtype)
    return fwd, bwd, size


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(H=3), INVALID), (dict(Hkv=0), INVALID), (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(dtype=3), INVALID), (dict(D=48), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(B=65535, Hkv=4, H=4), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED)])
def test_window_sizes(kw, code):
    assert window(**kw) == (code, code, code)


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(q=0), INVALID, INVALID), (dict(out=0), INVALID, INVALID), (dict(k=0x1008), MISALIGNED, MISALIGNED),
    (dict(lse=0x1002), MISALIGNED, MISALIGNED), (dict(impl=3), INVALID, INVALID), (dict(impl=6), INVALID, INVALID),
    (dict(impl=2, dtype=0), UNSUPPORTED, UNSUPPORTED),
    (dict(dq=0), None, INVALID), (dict(dv=0x1004), None, MISALIGNED), (dict(workspace=0), None, INVALID),
    (dict(workspace=0x1010), None, MISALIGNED), (dict(ws=100), None, INVALID)])
def test_window_pointers(kw, fwd, bwd):
    a, b, _ = window(**kw)
    assert (fwd is None or a == fwd) and b == bwd


def paged(S=2, T=4, max_q=2, H=4, Hkv=2, D=64, n_pages=9, page=16, max_pages=4, window=0, sinks=0, dtype=1, impl=0,
          weights=0x1000, lse=0x1000, q=0x1000, k=0x1000, table=0x1000, ws=1 << 40, workspace=0x1000):
    lib = bd.load_library()
    v = ctypes.c_void_p
    a = lib.longnet_paged_attn_fwd(v(q), v(k), P, P, v(lse), v(weights), P, P, v(table), T, S, max_q, H, Hkv, D, n_pages,
                                   page, max_pages, window, sinks, dtype, impl, v(workspace), ws, None)
    b = lib.longnet_paged_append(P, P, v(k), P, v(weights), P, P, v(table), T, S, Hkv, D, n_pages, page, max_pages, dtype,
                                 None)
    c = lib.longnet_paged_workspace_bytes(S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype, 1)
    return a, b, c


@pytest.mark.parametrize("kw,attn,append,size", [
    (dict(S=0), INVALID, INVALID, INVALID), (dict(T=-1), INVALID, INVALID, None), (dict(n_pages=0), INVALID, INVALID, None),
    (dict(page=12), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED), (dict(page=4), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED),
    (dict(page=512), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED), (dict(D=80), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED),
    (dict(S=65535), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED, UNSUPPORTED, UNSUPPORTED),
    (dict(H=3), INVALID, None, INVALID), (dict(max_q=0), INVALID, None, INVALID), (dict(window=-1), INVALID, None, INVALID),
    (dict(sinks=-1), INVALID, None, INVALID), (dict(dtype=5), INVALID, INVALID, INVALID), (dict(impl=5), INVALID, None, None),
    (dict(impl=6, dtype=0), UNSUPPORTED, None, None), (dict(impl=2, dtype=0), UNSUPPORTED, None, None),
    (dict(lse=0), INVALID, None, None), (dict(q=0), INVALID, None, None), (dict(k=0), INVALID, INVALID, None),
    (dict(k=0x1004), MISALIGNED, MISALIGNED, None), (dict(table=0x1002), MISALIGNED, MISALIGNED, None),
    (dict(workspace=0x1020), MISALIGNED, None, None)])
def test_paged(kw, attn, append, size):
    a, b, c = paged(**kw)
    assert a == attn and (append is None or b == append) and (size is None or c == size)


def evict(S=2, Hkv=2, D=64, n_pages=9, page=16, max_pages=4, n_out=8, max_out=2, budget=20, sinks=2, recent=3, dtype=1,
          kept=0x1000, k_out=0x1000):
    v = ctypes.c_void_p
    return bd.load_library().longnet_cache_evict(P, P, P, P, P, v(k_out), P, P, P, v(kept), P, S, Hkv, D, n_pages, page,
                                                 max_pages, n_out, max_out, budget, sinks, recent, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(budget=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(sinks=10, recent=11), INVALID),
    (dict(budget=33), INVALID), (dict(kept=0), INVALID), (dict(k_out=0x1008), MISALIGNED), (dict(n_out=0), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(D=24), UNSUPPORTED), (dict(dtype=9), INVALID)])
def test_evict(kw, code):
    assert evict(**kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_device():
    no = bd.LONGNET_ERR_NO_DEVICE
    fwd, bwd, size = window()
    assert (fwd, bwd) == (no, no) and size > 0
    a, b, c = paged()
    assert (a, b) == (no, no) and c >= 0
    assert evict() == no


def test_binding_refuses_other_tensors():
    q = torch.zeros((1, 8, 2, 16))
    with pytest.raises(ValueError):
        bd.window_attn(q, q, q, 4)  # not CUDA tensors
    with pytest.raises(ValueError):
        bd.paged_append(q[0], q[0], q, q, q, q, torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(bd.LongNetError):
        bd.longnet_window_bwd_workspace_bytes(1, 8, 3, 2, 16, 4, 0, torch.float32)


def test_few_token_workspace_is_bounded():
    """The scores kept for the weights: at most 256 MiB, or one sequence's, whatever the table's capacity; with a
    window, of what it reaches."""
    size = lambda *a, w=True: bd.longnet_paged_workspace_bytes(*a, torch.bfloat16, w)  # noqa: E731
    for S, max_q, H, Hkv in ((64, 1, 32, 8), (64, 4, 32, 8), (256, 4, 32, 8), (2000, 1, 16, 1)):
        plain = size(S, max_q, H, Hkv, 128, 64, 2048, 0, 0, w=False)
        assert 0 < size(S, max_q, H, Hkv, 128, 64, 2048, 0, 0) - plain <= (256 << 20) + 1024
        rows, seen = max_q * H // Hkv, (1024 + 4 + 3 * 64) + 64
        windowed = size(S, max_q, H, Hkv, 128, 64, 2048, 1024, 4) - size(S, max_q, H, Hkv, 128, 64, 2048, 1024, 4, w=False)
        assert windowed <= min(256 << 20, 4 * S * Hkv * rows * seen) + 1024
    # one sequence's scores always fit
    one = size(1, 4, 32, 8, 128, 256, 1 << 14, 0, 0)
    assert one >= 4 * 8 * 16 * (1 << 22) and size(9, 4, 32, 8, 128, 256, 1 << 14, 0, 0) < one + (1 << 26)


@pytest.mark.parametrize("kw", [dict(max_pages=1 << 60), dict(max_pages=(1 << 60) + 4), dict(n_pages=1 << 60),
                                dict(n_pages=1 << 62), dict(max_q=1 << 62), dict(max_q=(1 << 62) + 1)])
def test_sizes_whose_products_pass_64_bits(kw):
    """Counts of pages and tokens whose product with the page size or the heads is small again modulo 2^64."""
    a, b, c = paged(**kw)
    assert a == UNSUPPORTED and ("max_q" in kw or b == UNSUPPORTED) and ("n_pages" in kw or c == UNSUPPORTED)
    if "max_q" not in kw:
        assert evict(**kw) == UNSUPPORTED
        assert evict(**{{"max_pages": "max_out", "n_pages": "n_out"}[n]: x for n, x in kw.items()}) == UNSUPPORTED


def test_no_token_needs_no_rows():
    """T = 0: an empty tensor has no address, and none is needed, with weights or without."""
    ok = bd.LONGNET_OK if torch.cuda.is_available() else bd.LONGNET_ERR_NO_DEVICE
    for weights in (0, 0x1000):
        assert paged(T=0, q=0, lse=0, weights=weights)[:2] == (ok, ok)


def test_workspace_sizes_go_by_value():
    """A size given as a tensor, or a number whose value a program changes in place, is read anew."""
    n = torch.tensor(1)
    small = bd.longnet_paged_workspace_bytes(4, n, 8, 2, 64, 16, 64, 0, 0, torch.bfloat16)
    n.fill_(700)
    large = bd.longnet_paged_workspace_bytes(4, n, 8, 2, 64, 16, 64, 0, 0, torch.bfloat16)
    assert small == bd.longnet_paged_workspace_bytes(4, 1, 8, 2, 64, 16, 64, 0, 0, torch.bfloat16)
    assert large == bd.longnet_paged_workspace_bytes(4, 700, 8, 2, 64, 16, 64, 0, 0, torch.bfloat16) != small
    w = torch.tensor(10)
    sizes = []
    for x in (10, 4000):
        w.fill_(x)
        sizes.append(bd.longnet_window_bwd_workspace_bytes(1, 8000, 4, 2, 64, w, 70, torch.bfloat16))
        assert sizes[-1] == bd.longnet_window_bwd_workspace_bytes(1, 8000, 4, 2, 64, x, 70, torch.bfloat16)
    assert sizes[0] != sizes[1]
