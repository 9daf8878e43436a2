"""The measured cases of the paged-cache operators and of the sliding window
with first tokens: what is timed, in plain torch operations and through the
library.

Four operators that work together.  A model is trained under a causal sliding
window whose first few tokens stay visible to every query (`fwd`, `bwd`), and
served from a paged key/value cache: `plan` turns request lengths into page
tables, slots and offsets, `store` writes the new tokens' keys and values into
their slots, `paged` is the attention of the new tokens over the cache.

Plain forms compute in 32 bits and round once at the end; `exact` computes the
same in 64 bits from the definitions, one request or head at a time.
"""
import math
import random

import numpy as np
import torch

own = False  # set by the caller: True runs the library's operators

D = 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a step of eight decoding requests: only latency counts
        dict(name="plan_decode_b8", op="plan", B=8, ps=64, ctx_lo=100, ctx_hi=4000, new_lo=1,
             new_hi=1, ended=0, cols=64, mix=1),
        # a large server step: 512 requests, some decoding, some with a chunk of
        # their prompt, some that have ended and give their pages back
        dict(name="plan_mixed_b512", op="plan", B=512, ps=16, ctx_lo=0, ctx_hi=8000, new_lo=1,
             new_hi=64, ended=31, cols=520, mix=2),
        # one decode step of 32 requests
        dict(name="store_decode_t32", op="store", T=32, pad=0, Hkv=8, ps=64, layout="HND",
             dtype="bf16", pages=512),
        # a prefill chunk of 16384 tokens, padded by a few rows without a slot
        dict(name="store_chunk_t16384", op="store", T=16384, pad=77, Hkv=8, ps=16, layout="NHD",
             dtype="f16", pages=2048),
        # a single user's decode step at a short context: latency
        dict(name="paged_decode_one", op="paged", B=1, Hq=32, Hkv=8, ps=16, layout="NHD",
             dtype="f16", ctx_lo=1000, ctx_hi=1000, new_lo=1, new_hi=1, chunk=0, kind="causal",
             window=0, first=0, sink=False, mix=3),
        # a batch of decodes at ragged contexts: the cache's bandwidth
        dict(name="paged_decode_b64", op="paged", B=64, Hq=64, Hkv=8, ps=64, layout="HND",
             dtype="bf16", ctx_lo=2000, ctx_hi=16000, new_lo=1, new_hi=1, chunk=0, kind="causal",
             window=0, first=0, sink=True, mix=4),
        # two users at long contexts, a few speculated tokens each: one request's
        # keys have to be split over the GPU
        dict(name="paged_decode_long", op="paged", B=2, Hq=32, Hkv=4, ps=32, layout="HND",
             dtype="bf16", ctx_lo=60000, ctx_hi=130000, new_lo=3, new_hi=5, chunk=0,
             kind="causal", window=0, first=0, sink=False, mix=5),
        # chunks of two prompts over what is cached already: the tensor cores
        dict(name="paged_chunk_b2", op="paged", B=2, Hq=32, Hkv=8, ps=64, layout="HND",
             dtype="bf16", ctx_lo=7000, ctx_hi=9001, new_lo=1800, new_hi=2048, chunk=0,
             kind="causal", window=0, first=0, sink=False, mix=6),
        # a step of a model with a window and first tokens: decodes beside one chunk
        dict(name="paged_window_mixed", op="paged", B=16, Hq=32, Hkv=8, ps=32, layout="NHD",
             dtype="f16", ctx_lo=500, ctx_hi=16000, new_lo=1, new_hi=4, chunk=500,
             kind="first", window=1024, first=4, sink=True, mix=7),
        # the training forward at an ordinary size
        dict(name="window_fwd_s8192", op="fwd", B=1, Hq=32, Hkv=8, S=8192, window=1024, first=64,
             dtype="bf16", sink=True),
        # the training backward: a small odd size, and an ordinary one
        dict(name="window_bwd_s1000", op="bwd", B=2, Hq=8, Hkv=2, S=1000, window=128, first=5,
             dtype="f16", sink=True),
        dict(name="window_bwd_s8192", op="bwd", B=1, Hq=32, Hkv=8, S=8192, window=1024, first=4,
             dtype="bf16", sink=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "paged", "paged", "fwd", "bwd"])
    dtype = rng.choice(["f16", "bf16"])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        B, ps = _log(rng, 1, 512), rng.choice([16, 32, 48, 64, 128])
        hi, new = _log(rng, 16, 8000), _log(rng, 1, 64)
        return dict(op=op, B=B, ps=ps, ctx_lo=0, ctx_hi=hi, new_lo=0, new_hi=new,
                    ended=rng.randint(0, B // 8), cols=-(-(hi + new) // ps) + rng.randint(0, 9),
                    mix=mix)
    if op == "store":
        T, Hkv, ps = _log(rng, 1, 16384), rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 48, 64])
        return dict(op=op, T=T, pad=rng.randint(0, 100), Hkv=Hkv, ps=ps,
                    layout=rng.choice(["HND", "NHD"]), dtype=dtype,
                    pages=-(-T // ps) + rng.randint(1, 300))
    kind = rng.choice(["causal", "first", "first", "sliding"])
    window = _log(rng, 1, 4096)
    first = _log(rng, 1, 300) if kind == "first" else 0
    if op == "paged":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        # decode steps, speculated tokens, chunks: the longer the chunk the fewer requests
        new = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 8, 1000)])
        B = _log(rng, 1, 48 if new <= 8 else 6)
        hi = _log(rng, 64, 16000 if new <= 8 else 6000)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, ps=rng.choice([16, 32, 48, 64, 128]),
                    layout=rng.choice(["HND", "NHD"]), dtype=dtype, ctx_lo=1, ctx_hi=hi,
                    new_lo=1, new_hi=new, chunk=0, kind=kind,
                    window=window if kind != "causal" else 0, first=first,
                    sink=rng.random() < 0.5, mix=mix)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4])
    return dict(op=op, B=rng.choice([1, 1, 2]), Hq=Hq, Hkv=Hkv, S=_log(rng, 1, 5500),
                window=window, first=_log(rng, 1, 300), dtype=dtype, sink=rng.random() < 0.5)


def _lengths(case):
    """(new tokens, keys) of each request: they belong to the case, so that its
    work is known without its inputs."""
    r = random.Random(case["mix"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    if case["op"] == "plan":
        ended = set(r.sample(range(case["B"]), case["ended"]))
        old = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in new]
        return [-1 if b in ended else n for b, n in enumerate(new)], old
    if case["chunk"]:
        new[r.randrange(case["B"])] = case["chunk"]
    return new, [max(n, r.randint(case["ctx_lo"], case["ctx_hi"])) for n in new]


def _rule(case):
    """(window, first) of the causal rule: key j is visible to position i when
    j <= i and (i - j < window or j < first)."""
    if case["op"] in ("fwd", "bwd"):
        return case["window"], case["first"]
    return (case["window"] or 1 << 30), case["first"]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "plan":
        ps, (new, old) = case["ps"], _lengths(case)
        held = [-(-n // ps) for n in old]
        need = [max(0, -(-(o + n) // ps) - h) if n > 0 else 0 for n, o, h in zip(new, old, held)]
        pages = sum(held) + sum(need) + 16
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["B"], case["cols"]), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(case["cols"], device="cuda")[None, :]
        h = _ints(held).long()
        start = h.cumsum(0) - h
        table = torch.where(col < h[:, None],
                            perm[(start[:, None] + col).clamp(max=pages - 1)], table)
        free = torch.zeros(pages, dtype=torch.int32, device="cuda")
        n_free = pages - sum(held)
        free[:n_free] = perm[sum(held):]
        st.update(cached=_ints(old), fresh=_ints(new), free_pages=free,
                  free_count=_ints([n_free]), block_table=table, pages=pages,
                  tokens=sum(max(n, 0) for n in new) + 8)
        return st
    dt = DTYPES[case["dtype"]]
    if op == "store":
        T, pad, Hkv, ps, P = case["T"], case["pad"], case["Hkv"], case["ps"], case["pages"]
        shape = (P, Hkv, ps, D) if case["layout"] == "HND" else (P, ps, Hkv, D)
        st["k_pages"], st["v_pages"] = _normal(g, shape, dt), _normal(g, shape, dt)
        # keys and values as slices of a fused projection's output
        qkv = _normal(g, (T + pad, 3 * Hkv, D), dt)
        st["k"], st["v"] = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
        slot = torch.randperm(P * ps, generator=g, device="cuda")[:T]
        st["slot_map"] = torch.cat([slot, torch.full((pad,), -1, device="cuda",
                                                     dtype=torch.int64)])
        return st
    Hq, Hkv, B = case["Hq"], case["Hkv"], case["B"]
    sink = torch.randn(Hq, generator=g, device="cuda") if case["sink"] else None
    st["sink"], st["scale"] = sink, 1.0 / math.sqrt(D)
    if op == "paged":
        ps, (new, ctx) = case["ps"], _lengths(case)
        held = [-(-n // ps) for n in ctx]
        P = sum(held) + 7
        shape = (P, Hkv, ps, D) if case["layout"] == "HND" else (P, ps, Hkv, D)
        st["k_pages"], st["v_pages"] = _normal(g, shape, dt), _normal(g, shape, dt)
        perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        h = _ints(held).long()
        col = torch.arange(max(held) + 1, device="cuda")[None, :]
        start = h.cumsum(0) - h
        st["block_table"] = torch.where(col < h[:, None],
                                        perm[(start[:, None] + col).clamp(max=P - 1)],
                                        torch.full_like(perm[:1], -1))
        T = sum(new)
        st["q"] = _normal(g, (T, Hq, D), dt)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st.update(cu=_ints(cu), seqlen_k=_ints(ctx), T=T, max_q=max(new), max_k=max(ctx))
        return st
    S = case["S"]
    st["q"], st["k"] = _normal(g, (B, Hq, S, D), dt), _normal(g, (B, Hkv, S, D), dt)
    st["v"] = _normal(g, (B, Hkv, S, D), dt)
    if op == "bwd":
        # the forward's output and row statistics, as the training step has kept them
        st["dO"] = _normal(g, (B, Hq, S, D), dt)
        st["o"], st["lse"] = _plain_fwd(st)
    return st


# ------------------------------------------------------------------ plain forms

def _plain_plan(st):
    """In request order; ended requests give their pages back first."""
    case, ps = st["case"], st["case"]["ps"]
    cached, fresh = st["cached"].long(), st["fresh"].long()
    table, free = st["block_table"], st["free_pages"]
    B, cols = table.shape
    P, T = free.numel(), st["tokens"]
    live, new = fresh >= 0, fresh.clamp(min=0)
    held = (cached + ps - 1) // ps
    # ended requests: their pages onto the stack, in request order
    back = torch.where(live, 0, held)
    at = st["free_count"].long() + back.cumsum(0) - back
    col = torch.arange(cols, device=table.device)[None, :]
    dest = torch.where(col < back[:, None], at[:, None] + col, P)
    stack = torch.cat([free, free[:1]])
    stack[dest.reshape(-1)] = table.reshape(-1)
    free.copy_(stack[:P])
    count = st["free_count"].long() + back.sum()
    # the others: the pages their new tokens need, from the top of the stack
    need = torch.where(live, (cached + new + ps - 1) // ps - held, 0)
    upto = need.cumsum(0)
    end = new.cumsum(0)
    refused = live & (((need > 0) & (upto > count)) | (cached + new > cols * ps) | (end > T))
    grant = torch.where(refused, 0, need)
    j = col - held[:, None]
    take = (j >= 0) & (j < grant[:, None])
    top = (count - 1 - ((upto - need)[:, None] + j)).clamp(0, P - 1)
    table.copy_(torch.where(take, free[top], table))
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), end])
    seqlen = torch.where(live, torch.where(refused, cached, cached + new), 0)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    used = t < end[-1]
    pos = cached[b] + t - cu[b]
    ok = used & ~refused[b]
    page = table[b, (pos // ps).clamp(0, cols - 1)].long()
    slot = torch.where(ok, page * ps + pos % ps, -1)
    return dict(cu_seqlens_q=cu.int(), seqlen_k=seqlen.int(), block_table=table,
                free_pages=free, free_count=(count - grant.sum()).int().reshape(1),
                slot_map=slot, position=torch.where(used, pos, -1).int(),
                refused=refused.sum().int().reshape(1))


def _plain_store(st):
    ps, keep = st["case"]["ps"], st["slot_map"] >= 0
    slot = st["slot_map"][keep]
    page, row = slot // ps, slot % ps
    for pages, x in ((st["k_pages"], st["k"]), (st["v_pages"], st["v"])):
        if st["case"]["layout"] == "HND":
            pages[page, :, row] = x[keep]
        else:
            pages[page, row] = x[keep]
    return st["k_pages"], st["v_pages"]


def _softmax(s, sink, v):
    """exp, sums and the weighted values of masked scores s [..., g, n, l] against
    v [..., l, D]; sink [g, 1, 1]-shaped or None."""
    m = s.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == NEG, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    if sink is not None:
        l = l + torch.exp(sink - m)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    return o, torch.where(l > 0, m + torch.log(l), math.inf).squeeze(-1)


def _plain_paged(st):
    case = st["case"]
    ps, (window, first) = case["ps"], _rule(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    g, B = Hq // Hkv, case["B"]
    table = st["block_table"][:, :-(-st["max_k"] // ps)].long().clamp(min=0)
    Lp = table.shape[1] * ps

    def rows(pages):  # [B, Hkv, 1, Lp, D]
        x = pages[table]
        x = x if case["layout"] == "NHD" else x.transpose(2, 3)
        return x.reshape(B, Lp, Hkv, D).permute(0, 2, 1, 3).float().unsqueeze(2)

    cu, L = st["cu"].long(), st["seqlen_k"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(st["max_q"], device="cuda")
    tok = (cu[:-1, None] + i).clamp(max=st["T"] - 1)
    q = st["q"][tok].float().reshape(B, -1, Hkv, g, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q, rows(st["k_pages"]).transpose(-1, -2)) * st["scale"]
    pos = (L - n)[:, None, None] + i[None, :, None]
    j = torch.arange(Lp, device="cuda")[None, None, :]
    vis = (j <= pos) & (j < L[:, None, None]) & ((pos - j < window) | (j < first))
    s = torch.where(vis[:, None, None], s, NEG)
    sink = None if st["sink"] is None else st["sink"].reshape(Hkv, g, 1, 1)
    o, lse = _softmax(s, sink, rows(st["v_pages"]))
    # back to the packed rows of the new tokens
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, D)[b, t - cu[b]]
    lse = lse.permute(0, 3, 1, 2).reshape(B, -1, Hq)[b, t - cu[b]]
    return o.to(st["q"].dtype), lse.t().contiguous()


def _visible(case):
    window, first = _rule(case)
    i = torch.arange(case["S"], device="cuda")[:, None]
    j = torch.arange(case["S"], device="cuda")[None, :]
    return (j <= i) & ((i - j < window) | (j < first))


def _heads(case, x):
    """[B, H, S, D] as [B, Hkv, heads of the group, S, D] in 32 bits."""
    return x.float().reshape(case["B"], case["Hkv"], -1, case["S"], D)


def _plain_fwd(st):
    case = st["case"]
    q, k, v = (_heads(case, st[n]) for n in "qkv")
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    s = torch.where(_visible(case), s, NEG)
    sink = None if st["sink"] is None else st["sink"].reshape(case["Hkv"], -1, 1, 1)
    o, lse = _softmax(s, sink, v)
    shape = st["q"].shape
    return o.reshape(shape).to(st["q"].dtype), lse.reshape(shape[:3])


def _plain_bwd(st):
    case = st["case"]
    q, k, v, o, dO = (_heads(case, st[n]) for n in ("q", "k", "v", "o", "dO"))
    lse = st["lse"].reshape(case["B"], case["Hkv"], -1, case["S"], 1)
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    p = torch.where(_visible(case), torch.exp(s - lse), 0.0)
    delta = (dO * o).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), dO).sum(2)
    ds = p * (torch.matmul(dO, v.transpose(-1, -2)) - delta)
    dq = torch.matmul(ds, k) * st["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * st["scale"]
    dt = st["q"].dtype
    out = [dq.reshape(st["q"].shape).to(dt), dk.to(dt), dv.to(dt)]
    if st["sink"] is not None:
        sink = st["sink"].double().reshape(case["Hkv"], -1, 1, 1)
        ds = -(torch.exp(sink - lse.double()) * delta.double())
        out.append(ds.sum((0, 3, 4)).reshape(-1).float())
    return tuple(out)


# ------------------------------------------------------------------ one pass

def _own_run(st):
    from masked_attention_backward_gb300 import binding as mab
    case = st["case"]
    op = case["op"]
    if op == "plan":
        plan = mab.paged_plan(st["cached"], st["fresh"], st["free_pages"], st["free_count"],
                              st["block_table"], case["ps"], max_tokens=st["tokens"])
        return dict(cu_seqlens_q=plan.cu_seqlens_q, seqlen_k=plan.seqlen_k,
                    block_table=st["block_table"], free_pages=st["free_pages"],
                    free_count=plan.free_count, slot_map=plan.slot_map, position=plan.position,
                    refused=plan.refused)
    if op == "store":
        cache = mab.PagedCache(st["k_pages"], st["v_pages"], case["layout"])
        mab.paged_store(cache, st["k"], st["v"], st["slot_map"])
        return st["k_pages"], st["v_pages"]
    kind = {"causal": mab.ATTN_MASK_CAUSAL, "sliding": mab.ATTN_MASK_SLIDING,
            "first": mab.ATTN_MASK_SLIDING_FIRST}[case.get("kind", "first")]
    if op == "paged":
        cache = mab.PagedCache(st["k_pages"], st["v_pages"], case["layout"])
        mask = mab.Mask(kind=kind, window=case["window"], first=case["first"],
                        cu_seqlens_q=st["cu"], seqlen_k=st["seqlen_k"], max_seqlen_q=st["max_q"],
                        max_seqlen_k=st["max_k"], total_q=st["T"])
        return mab.paged_fwd(st["q"], cache, st["block_table"], st["sink"], mask, st["scale"])
    mask = mab.Mask(kind=kind, window=case["window"], first=case["first"])
    if op == "fwd":
        return mab.fwd(st["q"], st["k"], st["v"], st["sink"], mask, st["scale"])
    grads = mab.bwd(st["q"], st["k"], st["v"], st["o"], st["dO"], st["lse"], st["sink"], mask,
                    st["scale"])
    return grads if st["sink"] is not None else grads[:3]


def run(st):
    if own:
        return _own_run(st)
    return {"plan": _plain_plan, "store": _plain_store, "paged": _plain_paged,
            "fwd": _plain_fwd, "bwd": _plain_bwd}[st["case"]["op"]](st)


# ------------------------------------------------------------------ the work

def _pairs(positions, window, first):
    pos = np.asarray(positions, dtype=np.int64)
    return int((np.minimum(pos + 1, window) +
                np.clip(np.minimum(pos - window + 1, first), 0, None)).sum())


def work(case):
    op = case["op"]
    if op == "plan":
        ps, (new, old) = case["ps"], _lengths(case)
        T = sum(max(n, 0) for n in new)
        got = sum(max(0, -(-(o + n) // ps) + -o // ps) for n, o in zip(new, old) if n > 0)
        back = sum(-(-o // ps) for n, o in zip(new, old) if n < 0)
        # lengths in, offsets and lengths out, pages moved either way, slots and positions
        return {"bytes": 16 * case["B"] + 8 * (got + back) + 12 * T, "flops": 0}
    if op == "store":
        return {"bytes": case["T"] * (8 + 4 * case["Hkv"] * D * 2), "flops": 0}
    window, first = _rule(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "paged":
        new, ctx = _lengths(case)
        pairs = keys = 0
        for n, L in zip(new, ctx):
            pairs += _pairs(np.arange(L - n, L), window, first)
            lo = max(0, L - n - window + 1)
            keys += L - lo + min(first, lo)
        T = sum(new)
        return {"bytes": 2 * T * Hq * D * 2 + T * Hq * 4 + 2 * keys * Hkv * D * 2,
                "flops": 4 * D * pairs * Hq}
    B, S = case["B"], case["S"]
    pairs = B * Hq * _pairs(np.arange(S), window, first)
    rq, rk = B * Hq * S * D * 2, B * Hkv * S * D * 2
    if op == "fwd":
        return {"bytes": 2 * rq + 2 * rk + B * Hq * S * 4, "flops": 4 * D * pairs}
    return {"bytes": 4 * rq + 4 * rk + B * Hq * S * 4, "flops": 10 * D * pairs}


# ------------------------------------------------------------------ 64 bits

def _attend64(q, k, v, vis, sink, scale):
    """One head: rows q [n, D] over keys k, values v [l, D] under vis [n, l]."""
    s = (q.double() @ k.double().T * scale).masked_fill(~vis, NEG)
    if sink is not None:
        s = torch.cat([s, sink.double().expand(s.shape[0], 1)], 1)
    lse = torch.logsumexp(s, 1)
    seen = lse > NEG
    p = torch.exp(s - torch.where(seen, lse, 0.0)[:, None])[:, :k.shape[0]]
    return p @ v.double(), torch.where(seen, lse, math.inf)


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    st = prepare(case, seed)
    if op == "store":
        ps, slots = case["ps"], st["slot_map"].tolist()
        src = torch.tensor([t for t, s in enumerate(slots) if s >= 0], device="cuda")
        dst = torch.tensor([s for s in slots if s >= 0], device="cuda")
        out = []
        for pages, x in ((st["k_pages"], st["k"]), (st["v_pages"], st["v"])):
            y = pages.double()
            y = y.transpose(1, 2).contiguous() if case["layout"] == "HND" else y
            y.view(-1, case["Hkv"], D).index_copy_(0, dst, x.double().index_select(0, src))
            out.append(y.transpose(1, 2).contiguous() if case["layout"] == "HND" else y)
        return tuple(out)
    window, first = _rule(case)
    Hq, group = case["Hq"], case["Hq"] // case["Hkv"]
    if op == "paged":
        new, ctx = _lengths(case)
        o = torch.zeros(st["T"], Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(Hq, st["T"], dtype=torch.float64, device="cuda")
        t0 = 0
        for b, (n, L) in enumerate(zip(new, ctx)):
            ids = st["block_table"][b, :-(-L // case["ps"])].long()
            ks, vs = st["k_pages"][ids], st["v_pages"][ids]
            if case["layout"] == "HND":
                ks, vs = ks.transpose(1, 2), vs.transpose(1, 2)
            ks, vs = ks.flatten(0, 1)[:L], vs.flatten(0, 1)[:L]
            i = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None, :]
            vis = (i >= j) & ((j > i - window) | (j < first))
            for h in range(Hq):
                o[t0:t0 + n, h], lse[h, t0:t0 + n] = _attend64(
                    st["q"][t0:t0 + n, h], ks[:, h // group], vs[:, h // group], vis,
                    None if st["sink"] is None else st["sink"][h], st["scale"])
            t0 += n
        return o, lse
    B, S = case["B"], case["S"]
    i = torch.arange(S, device="cuda")[:, None]
    j = torch.arange(S, device="cuda")[None, :]
    vis = (i >= j) & ((j > i - window) | (j < first))
    z = dict(dtype=torch.float64, device="cuda")
    if op == "fwd":
        o, lse = torch.zeros(B, Hq, S, D, **z), torch.zeros(B, Hq, S, **z)
        for b in range(B):
            for h in range(Hq):
                o[b, h], lse[b, h] = _attend64(
                    st["q"][b, h], st["k"][b, h // group], st["v"][b, h // group], vis,
                    None if st["sink"] is None else st["sink"][h], st["scale"])
        return o, lse
    dq = torch.zeros(B, Hq, S, D, **z)
    dk, dv = torch.zeros(B, Hq // group, S, D, **z), torch.zeros(B, Hq // group, S, D, **z)
    dsink = torch.zeros(Hq, **z)
    for b in range(B):
        for h in range(Hq):
            c = h // group
            q, o, dO = (st[x][b, h].double() for x in ("q", "o", "dO"))
            k, v, lse = st["k"][b, c].double(), st["v"][b, c].double(), st["lse"][b, h].double()
            p = torch.exp(q @ k.T * st["scale"] - lse[:, None]).masked_fill(~vis, 0.0)
            delta = (dO * o).sum(1)
            ds = p * (dO @ v.T - delta[:, None])
            dq[b, h] = ds @ k * st["scale"]
            dk[b, c] += ds.T @ q * st["scale"]
            dv[b, c] += p.T @ dO
            if st["sink"] is not None:
                dsink[h] -= (torch.exp(st["sink"][h].double() - lse) * delta).sum()
    return (dq, dk, dv, dsink) if st["sink"] is not None else (dq, dk, dv)
