"""Plain 64-bit forms of the sliding-window and paged-cache operators, and the
error bounds of the kernels' roundings, for the tests."""
from __future__ import annotations

import math

import torch

# The size of one rounding, relative: half a step of the format.
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# fp32 arithmetic of a score: its D products and sums, the scale and the
# exponential, each 2^-24 relative to terms of a few units (the draws are
# N(0, 1)); e^s then carries it as a relative error.
FP32 = 4e-5
# A value below fp16's normal range is rounded to a multiple of 2^-24.
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def visible(x, j, window, sinks):
    see = j <= x
    return see & ((x - j < window) | (j < sinks)) if window else see


def attend(q, k, v, first, window, sinks):
    """q [n, D] at positions first.., k, v [m, D], float64 -> out, lse, P."""
    s = q @ k.T / math.sqrt(q.shape[1])
    x = torch.arange(first, first + q.shape[0], device=q.device)[:, None]
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    see = visible(x, j, window, sinks)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    p = torch.where(see, torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]),
                    torch.zeros_like(s))
    return p @ v, lse, p


def out_bound(p, v, out, dtype):
    """P rounded to the 16-bit format (relative), out rounded once, fp32 inside."""
    u, t = HALF[dtype], TINY[dtype]
    return u * out.abs() + (u + FP32) * (p @ v.abs()) + t * v.abs().sum(0) + 1e-6


def window_reference(q, k, v, dout, window, sinks):
    """[B, N, H, D] inputs -> (out, lse, dq, dk, dv) and their bounds, float64."""
    B, N, H, D = q.shape
    Hkv = k.shape[2]
    G, sc, dt = H // Hkv, 1 / math.sqrt(D), q.dtype
    u, t = HALF[dt], TINY[dt]
    q, k, v, dout = (z.double() for z in (q, k, v, dout))
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(k)
    lse = torch.zeros((B, H, N), dtype=torch.float64, device=q.device)
    b_out, b_dq, b_dk, b_dv = (torch.zeros_like(z) for z in (out, dq, dk, dv))
    for b in range(B):
        for h in range(H):
            f = h // G
            qq, kk, vv, do = q[b, :, h], k[b, :, f], v[b, :, f], dout[b, :, h]
            o, l, p = attend(qq, kk, vv, 0, window, sinks)
            out[b, :, h], lse[b, h] = o, l
            b_out[b, :, h] = out_bound(p, vv, o, dt)
            delta = (do * o).sum(-1, keepdim=True)
            dp = do @ vv.T
            ds = p * (dp - delta)
            # dS: rounded once; delta taken from the rounded out; P and dP in fp32
            off = (do.abs() * b_out[b, :, h]).sum(-1, keepdim=True)
            e_ds = u * ds.abs() + p * (off + FP32 * (do.abs() @ vv.abs().T + delta.abs())) + t
            dq[b, :, h] = ds @ kk * sc
            dk[b, :, f] += ds.T @ qq * sc
            dv[b, :, f] += p.T @ do
            b_dq[b, :, h] = e_ds @ kk.abs() * sc
            b_dk[b, :, f] += e_ds.T @ qq.abs() * sc
            b_dv[b, :, f] += ((u + FP32) * p + t).T @ do.abs()
    for g, bound in ((dq, b_dq), (dk, b_dk), (dv, b_dv)):
        bound += u * g.abs() + 1e-6
    return (out, lse, dq, dk, dv), (b_out, torch.full_like(lse, 1e-4), b_dq, b_dk, b_dv)


def within(name, got, ref, bound):
    d = (got.double() - ref).abs()
    ok = d <= bound * 1.001
    same = (got.double() == ref) | (got.double().isnan() & ref.isnan())  # infinities
    assert bool((ok | same).all()), (
        f"{name}: {int((~(ok | same)).sum())} of {ok.numel()} values out of bounds, worst {float(d[~(ok | same)].max())} "
        f"against {float(bound.max())}")


class Cache:
    """A paged cache with shuffled pages, NaN in every slot no key uses, and
    page numbers out of range in the table where no key is."""

    def __init__(self, lens, page, Hkv, D, dtype, seed, spare=4, wide=None, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.page, self.Hkv, self.D, self.dtype = page, Hkv, D, dtype
        S = len(lens)
        wide = wide or max(1, max(-(-n // page) for n in lens))
        n_pages = sum(-(-n // page) for n in lens) + spare
        order = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((S, wide), -7, dtype=torch.int32)
        self.k = [torch.randn((n, Hkv, D), generator=g).to(dtype).to(device) for n in lens]
        self.v = [torch.randn((n, Hkv, D), generator=g).to(dtype).to(device) for n in lens]
        self.k_pages = torch.full((n_pages, page, Hkv, D), float("nan"), dtype=dtype, device=device)
        self.v_pages = torch.full_like(self.k_pages, float("nan"))
        for s, n in enumerate(lens):
            for i in range(-(-n // page)):
                pg = order.pop()
                table[s, i] = pg
                m = min(page, n - i * page)
                self.k_pages[pg, :m] = self.k[s][i * page:i * page + m]
                self.v_pages[pg, :m] = self.v[s][i * page:i * page + m]
        self.free = order
        self.table = table.to(device)
        self.lens = list(lens)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)


def paged_reference(cache, q, nq, window, sinks):
    """q [T, H, D] packed -> out, lse, weights received and the bounds of out and weights."""
    T, H, D = q.shape
    Hkv = cache.Hkv
    G = H // Hkv
    out = torch.zeros((T, H, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((T, H), dtype=torch.float64, device=q.device)
    b_out = torch.zeros_like(out)
    w = torch.zeros((len(nq), Hkv, cache.table.shape[1] * cache.page), dtype=torch.float64, device=q.device)
    at = 0
    for s, n in enumerate(nq):
        if n:
            m = cache.lens[s]
            for h in range(H):
                f = h // G
                kk, vv = cache.k[s][:, f].double(), cache.v[s][:, f].double()
                o, l, p = attend(q[at:at + n, h].double(), kk, vv, m - n, window, sinks)
                out[at:at + n, h], lse[at:at + n, h] = o, l
                b_out[at:at + n, h] = out_bound(p, vv, o, q.dtype)
                w[s, f, :m] += p.sum(0)
        at += n
    return out, lse, w, b_out


def evict_reference(weights, lens, budget, sinks, recent):
    """kept indices of each (sequence, head), by sorting on the CPU."""
    S, Hkv, _ = weights.shape
    kept = torch.full((S, Hkv, budget), -1, dtype=torch.int64)
    for s, n in enumerate(lens):
        for f in range(Hkv):
            if n <= budget:
                sel = list(range(n))
            else:
                w = weights[s, f].tolist()
                mid = sorted(range(sinks, n - recent), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0, j))
                sel = sorted(list(range(sinks)) + mid[:budget - sinks - recent] + list(range(n - recent, n)))
            kept[s, f, :len(sel)] = torch.tensor(sel, dtype=torch.int64)
    return kept
