"""Cases of the sliding-window and paged-cache attention operators.

Three paths of a program that trains and serves a causal attention layer:

  train   one layer's attention with a sliding window and a few first tokens
          that stay visible, forward and backward;
  serve   one step over a paged key/value cache: the new tokens' keys and
          values are appended, then the new tokens attend to the cache
          (single tokens or chunks of a prompt), with or without the sum of
          the attention weights that each cached key received;
  evict   the cache of each sequence cut down to a budget of keys: the first,
          the latest and those that received most attention weight.

Definitions.  Query head h reads key/value head h // (H / Hkv).  The query at
position x sees key j when j <= x and (window == 0 or x - j < window or
j < sinks); scores are <q, k> / sqrt(D).  A row that sees nothing has out = 0
and lse = -inf.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest training call: launch latency
        dict(name="train_tiny_bf16", kind="train", B=2, N=128, H=4, Hkv=2, D=64, window=64, sinks=4, dtype="bf16"),
        # full-precision training at an odd length, narrow heads
        dict(name="train_odd_fp32", kind="train", B=1, N=997, H=6, Hkv=2, D=32, window=200, sinks=3, dtype="fp32"),
        # a language-model layer at 8K tokens, shared key/value heads
        dict(name="train_lm_bf16", kind="train", B=1, N=8192, H=12, Hkv=4, D=64, window=1024, sinks=4,
             dtype="bf16"),
        # long-sequence training with wide heads and a wide window
        dict(name="train_long_fp16", kind="train", B=1, N=16384, H=8, Hkv=8, D=128, window=4096, sinks=16,
             dtype="fp16"),
        # one user, one token, a short context: latency
        dict(name="decode_one_bf16", kind="serve", S=1, max_q=1, kv=500, H=12, Hkv=12, D=64, page=16, window=0,
             sinks=0, weights=False, pad=0, dtype="bf16"),
        # a full serving batch generating, contexts of all lengths, weights kept for eviction
        dict(name="decode_batch_weights", kind="serve", S=64, max_q=1, kv=8192, H=32, Hkv=8, D=128, page=64,
             window=0, sinks=0, weights=True, pad=3, dtype="bf16"),
        # few users with very long contexts: the cache has to be split over the GPU
        dict(name="decode_long_fp16", kind="serve", S=4, max_q=1, kv=131072, H=16, Hkv=2, D=128, page=128, window=0,
             sinks=0, weights=False, pad=0, dtype="fp16"),
        # a mixed batch: single tokens and chunks of several lengths, sliding window with sinks
        dict(name="chunk_mixed_window", kind="serve", S=7, max_q=700, kv=5000, H=12, Hkv=4, D=64, page=16,
             window=1024, sinks=4, weights=False, pad=5, dtype="fp16"),
        # chunks of long prompts
        dict(name="chunk_prompt_bf16", kind="serve", S=2, max_q=4096, kv=16384, H=16, Hkv=4, D=128, page=64,
             window=0, sinks=0, weights=False, pad=0, dtype="bf16"),
        # chunks of prompts that gather the weights for a later eviction
        dict(name="chunk_weights_bf16", kind="serve", S=3, max_q=1024, kv=8192, H=8, Hkv=2, D=128, page=32,
             window=0, sinks=0, weights=True, pad=0, dtype="bf16"),
        # a few short caches
        dict(name="evict_small", kind="evict", S=3, Hkv=4, D=64, page=16, kv=400, budget=128, sinks=4, recent=32,
             dtype="fp16"),
        # a serving batch's long caches cut to a quarter
        dict(name="evict_large", kind="evict", S=16, Hkv=8, D=128, page=64, kv=32768, budget=8192, sinks=4,
             recent=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["train", "train", "serve", "serve", "serve", "evict"])
    D = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "train":
        if rng.random() < 0.25:
            dtype = "fp32"
        Hkv = rng.choice([1, 2, 3, 4, 8])
        H = Hkv * rng.choice([1, 2, 3, 4])
        N = _log(rng, 1, 2048 if dtype == "fp32" else 8192)
        while H > Hkv and H * N * N > 8 * 8192 * 8192:
            H -= Hkv
        return dict(kind=kind, B=1 if N > 2048 else rng.choice([1, 2, 3]), N=N, H=H, Hkv=Hkv, D=D,
                    window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 65, 130]), dtype=dtype)
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if kind == "serve":
        H = Hkv * rng.choice([1, 2, 3, 4, 8])
        if rng.random() < 0.5:  # generation
            S, max_q = _log(rng, 1, 48), rng.choice([1, 1, 1, 2, 4])
            kv = _log(rng, max_q, max(max_q, min(65536, 300000 // S)))
        else:  # prompts
            S, max_q = rng.randint(1, 4), _log(rng, 5, 2048)
            kv = max_q + _log(rng, 1, 6000)
            while H > Hkv and S * H * max_q * kv * D > 2 * 16 * 4096 * 14336 * 128:
                H -= Hkv
        window = _log(rng, 1, 4096) if rng.random() < 0.4 else 0
        return dict(kind=kind, S=S, max_q=max_q, kv=kv, H=H, Hkv=Hkv, D=D, page=page, window=window,
                    sinks=rng.choice([1, 4, 70]) if window else 0, weights=rng.random() < 0.4,
                    pad=rng.choice([0, 0, 7]), dtype=dtype)
    S = _log(rng, 1, 16)
    kv = _log(rng, 3, 32768)
    budget = max(1, int(kv * rng.uniform(0.1, 1.1)))
    sinks = min(rng.choice([0, 4]), budget)
    return dict(kind=kind, S=S, Hkv=Hkv, D=D, page=page, kv=kv, budget=budget, sinks=sinks,
                recent=int((budget - sinks) * rng.choice([0, 0.1, 0.5, 1.0])), dtype=dtype)


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence: the longest first, the
    others spread below it; from the fifth on, every seventh is an idle slot."""
    r = random.Random("%d %d %d" % (c["S"], c.get("max_q", 0), c["kv"]))
    nq, kv = [], []
    for s in range(c["S"]):
        if s == 0:
            n, m = c.get("max_q", 0), c["kv"]
        elif s % 7 == 4:
            n, m = 0, 0
        else:
            n = r.randint(1, c["max_q"]) if c.get("max_q", 0) else 0
            if s % 3 == 2 and n:
                n = 1
            m = r.randint(max(n, c["kv"] // 4, 1), c["kv"])
        nq.append(n)
        kv.append(m)
    return nq, kv


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def _table(g, counts, page, width):
    """A page table [S, width] over a shuffled pool: -1 where a sequence has no page."""
    need = [-(-n // page) for n in counts]
    pages = max(1, sum(need)) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    rows, at = [], 0
    for n in need:
        rows.append(torch.cat([order[at:at + n], torch.full((width - n,), -1, dtype=torch.int32, device="cuda")]))
        at += n
    return torch.stack(rows).contiguous(), pages


def _weights(g, shape):
    """Accumulated attention weights: a heavy tail, and a share of keys that received none."""
    w = torch.exp(2 * torch.randn(shape, generator=g, device="cuda"))
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.2, torch.zeros_like(w), w)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _DT[c["dtype"]]
    if c["kind"] == "train":
        B, N, H, Hkv, D = (c[x] for x in ("B", "N", "H", "Hkv", "D"))
        return dict(c=c, q=_normal(g, (B, N, H, D), dt), k=_normal(g, (B, N, Hkv, D), dt),
                    v=_normal(g, (B, N, Hkv, D), dt), dout=_normal(g, (B, N, H, D), dt))
    S, Hkv, D, page = (c[x] for x in ("S", "Hkv", "D", "page"))
    nq, kv = _lengths(c)
    width = -(-c["kv"] // page)
    table, pages = _table(g, kv, page, width)
    st = dict(c=c, table=table, kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"),
              k_pages=_normal(g, (pages, page, Hkv, D), dt), v_pages=_normal(g, (pages, page, Hkv, D), dt))
    if c["kind"] == "evict":
        wide = -(-c["budget"] // page)
        new_table, new_pages = _table(g, [min(n, c["budget"]) for n in kv], page, wide)
        st.update(weights=_weights(g, (S, Hkv, width * page)), new_table=new_table,
                  k_new=torch.zeros((new_pages, page, Hkv, D), dtype=dt, device="cuda"),
                  v_new=torch.zeros((new_pages, page, Hkv, D), dtype=dt, device="cuda"))
        return st
    total = sum(nq)
    T, H = total + c["pad"], c["H"]
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    st.update(cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), total=total,
              q=_normal(g, (T, H, D), dt), k_tok=_normal(g, (T, Hkv, D), dt), v_tok=_normal(g, (T, Hkv, D), dt),
              out=torch.zeros((T, H, D), dtype=dt, device="cuda"),
              lse=torch.zeros((T, H), dtype=torch.float32, device="cuda"),
              weights=_weights(g, (S, Hkv, width * page)) if c["weights"] else None)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["c"]
    if c["kind"] == "train":
        if own:
            from sparse_long_sequence_attn_b200 import binding as bd

            out, lse = bd.window_attn(st["q"], st["k"], st["v"], c["window"], c["sinks"])
            dq, dk, dv = bd.window_attn_bwd(st["q"], st["k"], st["v"], out, lse, st["dout"], c["window"],
                                            c["sinks"])
            return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
        return _plain_train(c, st["q"], st["k"], st["v"], st["dout"])
    if c["kind"] == "serve":
        if own:
            from sparse_long_sequence_attn_b200 import binding as bd

            bd.paged_append(st["k_tok"], st["v_tok"], st["k_pages"], st["v_pages"], st["cu_q"], st["kv_len"],
                            st["table"], weights=st["weights"])
            bd.paged_attn(st["q"], st["k_pages"], st["v_pages"], st["cu_q"], st["kv_len"], st["table"], c["max_q"],
                          window=c["window"], sinks=c["sinks"], weights=st["weights"], out=st["out"], lse=st["lse"])
        else:
            _plain_serve(c, st)
        got = dict(out=st["out"], lse=st["lse"], k_pages=st["k_pages"], v_pages=st["v_pages"])
        if c["weights"]:
            got["weights"] = st["weights"]
        return got
    if own:
        from sparse_long_sequence_attn_b200 import binding as bd

        kept, new_len, new_weights = bd.cache_evict(
            st["k_pages"], st["v_pages"], st["weights"], st["kv_len"], st["table"], st["k_new"], st["v_new"],
            st["new_table"], c["budget"], sinks=c["sinks"], recent=c["recent"])
        return dict(kept=kept, new_len=new_len, new_weights=new_weights, k_new=st["k_new"], v_new=st["v_new"])
    return _plain_evict(c, st)


# ------------------------------------------------------------------ plain forms
def _visible(x, j, window, sinks):
    see = j <= x
    return see & ((x - j < window) | (j < sinks)) if window else see


def _plain_train(c, q, k, v, dout):
    B, N, H, Hkv, D = (c[x] for x in ("B", "N", "H", "Hkv", "D"))
    G, scale, dt = H // Hkv, 1.0 / math.sqrt(D), q.dtype
    heads = lambda t: t.float().permute(0, 2, 1, 3)  # noqa: E731
    qf, df = heads(q), heads(dout)
    kf, vf = (heads(t).repeat_interleave(G, 1) for t in (k, v))
    i = torch.arange(N, device=q.device)
    s = (qf @ kf.transpose(-1, -2)) * scale
    s.masked_fill_(~_visible(i[:, None], i[None, :], c["window"], c["sinks"]), float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p = p.div_(z)
    lse = (m + z.log())[..., 0]
    out = p @ vf
    dv = p.transpose(-1, -2) @ df
    dp = df @ vf.transpose(-1, -2)
    delta = (out * df).sum(-1, keepdim=True)
    ds = dp.sub_(delta).mul_(p)
    dq = (ds @ kf) * scale
    dk = (ds.transpose(-1, -2) @ qf) * scale
    back = lambda t: t.permute(0, 2, 1, 3).to(dt).contiguous()  # noqa: E731
    shared = lambda t: t.view(B, Hkv, G, N, D).sum(2)  # noqa: E731
    return dict(out=back(out), lse=lse, dq=back(dq), dk=back(shared(dk)), dv=back(shared(dv)))


def _plain_serve(c, st):
    S, H, Hkv, D, page, max_q = (c[x] for x in ("S", "H", "Hkv", "D", "page", "max_q"))
    G, scale = H // Hkv, 1.0 / math.sqrt(D)
    q, cu, kv, table = st["q"], st["cu_q"].long(), st["kv_len"].long(), st["table"].long()
    T, total, K = q.shape[0], st["total"], table.shape[1] * page
    nq = cu[1:] - cu[:-1]
    t = torch.arange(T, device=q.device)
    s_of = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=S - 1)  # the sequence of each row
    i_of = t - cu[s_of]
    pos = kv[s_of] - nq[s_of] + i_of
    # append
    at = pos[:total]
    where = (table[s_of[:total], at // page], at % page)
    st["k_pages"][where] = st["k_tok"][:total]
    st["v_pages"][where] = st["v_tok"][:total]
    if c["weights"]:  # a new key has received no weight yet
        st["weights"][s_of[:total], :, at] = 0.0
    # attend, all sequences padded to max_q queries and K keys
    flat = table.clamp(min=0)
    k = st["k_pages"][flat].view(S, K, Hkv, D).float().permute(0, 2, 1, 3)
    v = st["v_pages"][flat].view(S, K, Hkv, D).float().permute(0, 2, 1, 3)
    i = torch.arange(max_q, device=q.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=max(T - 1, 0))
    qp = q[rows].float().view(S, max_q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * max_q, D)
    x = (kv - nq)[:, None] + i[None, :]
    j = torch.arange(K, device=q.device)
    see = _visible(x[:, :, None], j, c["window"], c["sinks"]) & (i[None, :, None] < nq[:, None, None])
    see = see[:, None, None]
    sc = (qp @ k.transpose(-1, -2)).view(S, Hkv, G, max_q, K) * scale
    sc.masked_fill_(~see, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(z > 0, z, torch.ones_like(z)))
    lse = (m + z.log())[..., 0].permute(0, 3, 1, 2).reshape(S, max_q, H)
    if c["weights"]:
        st["weights"].add_(p.sum((2, 3)))
    o = (p.view(S, Hkv, G * max_q, K) @ v).view(S, Hkv, G, max_q, D).permute(0, 3, 1, 2, 4).reshape(S, max_q, H, D)
    i_at = i_of.clamp(0, max_q - 1)
    st["out"][:total] = o[s_of, i_at][:total].to(q.dtype)
    st["lse"][:total] = lse[s_of, i_at][:total]


def _plain_evict(c, st):
    S, Hkv, page, budget = (c[x] for x in ("S", "Hkv", "page", "budget"))
    w, kv, table, new_table = st["weights"], st["kv_len"].long(), st["table"].long(), st["new_table"].long()
    K, dev = w.shape[2], w.device
    j = torch.arange(K, device=dev)
    inside = (j[None, :] < kv[:, None])[:, None, :]
    always = ((j[None, :] < c["sinks"]) | (j[None, :] >= kv[:, None] - c["recent"]))[:, None, :] & inside
    inf = torch.full_like(w, float("inf"))
    rank = torch.where(always, inf, torch.where(inside, w, -inf))
    b = min(budget, K)
    top = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :b]
    new_len = kv.clamp(max=budget)
    n = torch.arange(budget, device=dev)
    live = (n[None, :] < new_len[:, None])[:, None, :].expand(S, Hkv, budget)
    kept = torch.full((S, Hkv, budget), K, dtype=torch.int64, device=dev)
    kept[..., :b] = torch.where(live[..., :b], top, kept[..., :b])
    kept = torch.sort(kept, dim=-1).values
    src = torch.where(live, kept, torch.zeros_like(kept))
    new_w = torch.zeros((S, Hkv, new_table.shape[1] * page), device=dev)
    new_w[..., :budget] = torch.where(live, torch.gather(w, 2, src), new_w[..., :budget])
    s_at, h_at, n_at = torch.nonzero(live, as_tuple=True)
    from_j = src[s_at, h_at, n_at]
    a, b_ = table[s_at, from_j // page], from_j % page
    x, y = new_table[s_at, n_at // page], n_at % page
    st["k_new"][x, y, h_at] = st["k_pages"][a, b_, h_at]
    st["v_new"][x, y, h_at] = st["v_pages"][a, b_, h_at]
    kept = torch.where(live, kept, torch.full_like(kept, -1))
    return dict(kept=kept.int(), new_len=new_len.int(), new_weights=new_w, k_new=st["k_new"], v_new=st["v_new"])


# ------------------------------------------------------------------ counts
def _seen(nq, kv, window, sinks):
    """(query, key) pairs that one head computes, and the keys that any query of the sequence sees."""
    first = kv - nq
    if not nq:
        return 0, 0
    if not window:
        return sum(range(first + 1, kv + 1)), kv
    pairs = sum(min(x + 1, window) + max(0, min(sinks, x + 1 - window)) for x in range(first, kv))
    low = max(0, first - window + 1)
    return pairs, kv - low + min(low, sinks)


def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    if c["kind"] == "train":
        B, N, H, Hkv, D = (c[x] for x in ("B", "N", "H", "Hkv", "D"))
        pairs, _ = _seen(N, N, c["window"], c["sinks"])
        # read q, k, v, dout; write out, lse, dq, dk, dv; two products forward, five backward
        return {"bytes": B * N * D * e * (4 * H + 4 * Hkv) + 4 * B * N * H, "flops": 7 * 2 * D * pairs * B * H}
    nq, kv = _lengths(c)
    if c["kind"] == "serve":
        H, Hkv, D = c["H"], c["Hkv"], c["D"]
        pairs = keys = 0
        for n, m in zip(nq, kv):
            p, k = _seen(n, m, c["window"], c["sinks"])
            pairs, keys = pairs + p, keys + k
        new = sum(nq)
        b = 2 * keys * Hkv * D * e  # the keys and values that are seen
        b += new * (2 * H * D * e + 4 * H) + 2 * new * Hkv * D * e  # q, out, lse; the new keys and values written
        if c["weights"]:
            b += 8 * keys * Hkv
        return {"bytes": b, "flops": 4 * D * pairs * H}
    left = sum(min(n, c["budget"]) for n in kv)
    # the weights read once, the kept rows read and written, the list of them and their weights written
    return {"bytes": 4 * sum(kv) * c["Hkv"] + left * c["Hkv"] * (4 * c["D"] * e + 8), "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(q, k, v, first, window, sinks):
    """q [G, n, D] at positions first.., k, v [m, D], all float64: out, lse and the weights."""
    s = torch.einsum("gnd,md->gnm", q, k) / math.sqrt(q.shape[-1])
    x = torch.arange(first, first + q.shape[1], device=q.device).view(1, -1, 1)
    j = torch.arange(k.shape[0], device=q.device).view(1, 1, -1)
    hidden = j > x
    if window:
        hidden = hidden | ((x - j >= window) & (j >= sinks))
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.unsqueeze(-1))
    return torch.einsum("gnm,md->gnd", p, v), lse, p


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["kind"] == "train":
        B, N, H, Hkv, D = (c[x] for x in ("B", "N", "H", "Hkv", "D"))
        G, scale = H // Hkv, 1.0 / math.sqrt(D)
        q, k, v, do = (st[x] for x in ("q", "k", "v", "dout"))
        out, dq = (torch.empty((B, N, H, D), dtype=torch.float64, device="cuda") for _ in range(2))
        dk, dv = (torch.zeros((B, N, Hkv, D), dtype=torch.float64, device="cuda") for _ in range(2))
        lse = torch.empty((B, H, N), dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(H):
                f = h // G
                qh, kh, vh, dh = q[b, :, h].double(), k[b, :, f].double(), v[b, :, f].double(), do[b, :, h].double()
                o, l, p = _exact_rows(qh[None], kh, vh, 0, c["window"], c["sinks"])
                out[b, :, h], lse[b, h] = o[0], l[0]
                p = p[0]
                dv[b, :, f] += torch.einsum("nm,nd->md", p, dh)
                g = torch.einsum("nd,md->nm", dh, vh)
                g = p * (g - (p * g).sum(-1, keepdim=True))
                dq[b, :, h] = torch.einsum("nm,md->nd", g, kh) * scale
                dk[b, :, f] += torch.einsum("nm,nd->md", g, qh) * scale
        return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
    if c["kind"] == "evict":
        kv, table, new_table = st["kv_len"].tolist(), st["table"].tolist(), st["new_table"].tolist()
        page, w = c["page"], st["weights"].double()
        new_w = torch.zeros((c["S"], c["Hkv"], len(new_table[0]) * page), dtype=torch.float64, device="cuda")
        kept = torch.full((c["S"], c["Hkv"], c["budget"]), -1, dtype=torch.int32, device="cuda")
        k_new, v_new = st["k_new"].double(), st["v_new"].double()
        for s, n in enumerate(kv):
            left = min(n, c["budget"])
            if not left:
                continue
            row = torch.tensor([x for x in table[s] if x >= 0], device="cuda")
            to = torch.tensor([x for x in new_table[s] if x >= 0], device="cuda")
            for h in range(c["Hkv"]):
                if n <= c["budget"]:
                    sel = torch.arange(n, device="cuda")
                else:
                    low, high = c["sinks"], n - c["recent"]
                    mid = w[s, h, low:high]
                    room = left - low - c["recent"]
                    best = torch.argsort(-mid, stable=True)[:room] + low
                    sel = torch.cat([torch.arange(low, device="cuda"), best.sort().values,
                                     torch.arange(high, n, device="cuda")])
                kept[s, h, :left] = sel.int()
                new_w[s, h, :left] = w[s, h, sel]
                d = torch.arange(left, device="cuda")
                k_new[to[d // page], d % page, h] = st["k_pages"][row[sel // page], sel % page, h].double()
                v_new[to[d // page], d % page, h] = st["v_pages"][row[sel // page], sel % page, h].double()
        return dict(kept=kept, new_len=st["kv_len"].clamp(max=c["budget"]), new_weights=new_w, k_new=k_new,
                    v_new=v_new)
    nq, kv = _lengths(c)
    page, G = c["page"], c["H"] // c["Hkv"]
    out, lse = st["out"].double(), st["lse"].double()
    weights = st["weights"].double() if c["weights"] else None
    at = 0
    for s, (n, m) in enumerate(zip(nq, kv)):
        if not n:
            continue
        row = st["table"][s, :-(-m // page)].long()
        x = torch.arange(m - n, m, device="cuda")
        st["k_pages"][row[x // page], x % page] = st["k_tok"][at:at + n]
        st["v_pages"][row[x // page], x % page] = st["v_tok"][at:at + n]
        if c["weights"]:
            weights[s, :, m - n:m] = 0
        kk, vv = (st[p][row].reshape(-1, c["Hkv"], c["D"])[:m].double() for p in ("k_pages", "v_pages"))
        for f in range(c["Hkv"]):
            qq = st["q"][at:at + n, f * G:(f + 1) * G].double().transpose(0, 1)
            o, l, p = _exact_rows(qq, kk[:, f], vv[:, f], m - n, c["window"], c["sinks"])
            out[at:at + n, f * G:(f + 1) * G] = o.transpose(0, 1)
            lse[at:at + n, f * G:(f + 1) * G] = l.transpose(0, 1)
            if c["weights"]:
                weights[s, f, :m] += p.sum((0, 1))
        at += n
    got = dict(out=out, lse=lse, k_pages=st["k_pages"].double(), v_pages=st["v_pages"].double())
    if c["weights"]:
        got["weights"] = weights
    return got
