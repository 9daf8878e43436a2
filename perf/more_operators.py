"""The measured cases of rotary positions and of the 8-bit paged cache: what is
timed, in plain torch operations and through the library.

Four operators of one serving step, of which the first is a training step's
too.  `rope` turns queries and keys by their positions (forward, and the
gradient's way back), `store` quantises the new tokens' keys and values into
their slots and reads the written blocks back, `load` reads whole prefixes back,
`paged` is the attention of the new tokens over the 8-bit cache.

The cache holds codes (e4m3, or int8 from -127 to 127) and one byte s a block of
tokens and key/value head: a value is code * 2^(s - 127).  A block's exponent is
the least for which its largest magnitude fits the codes.

Plain forms compute in 32 bits (angles in 64) and round once at the end; `exact`
computes the same in 64 bits from the definitions.
"""
import math
import random

import numpy as np
import torch

own = False  # set by the caller: True runs the library's operators

D = 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
TOP = {"e4m3": 448.0, "i8": 127.0}
# the least exponent of a block: below it the codes' values have no 16-bit form
LEAST = {("e4m3", "f16"): -15, ("i8", "f16"): -24, ("e4m3", "bf16"): -110, ("i8", "bf16"): -110}
NEG = float("-inf")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of eight requests far into their contexts, q and k slices of
        # one projection's output: only latency counts
        dict(name="rope_decode_t8", op="rope", back=False, layout="rows", B=1, S=8, Hq=32, Hkv=8,
             dtype="bf16", rot=128, interleaved=False, base=500000.0, scaling="none",
             far=1000000),
        # a training step's forward at an ordinary size, positions counted
        dict(name="rope_train_s8192", op="rope", back=False, layout="heads", B=1, S=8192, Hq=32,
             Hkv=8, dtype="bf16", rot=128, interleaved=False, base=10000.0, scaling="none", far=0),
        # the gradients of packed sequences: interleaved pairs, half of the head, scaled
        dict(name="rope_bwd_packed", op="rope", back=True, layout="rows", B=1, S=5003, Hq=24,
             Hkv=8, dtype="f16", rot=64, interleaved=True, base=10000.0, scaling="parts",
             far=30000),
        # one decode step of 32 requests: most blocks hold earlier tokens
        dict(name="store8_decode_t32", op="store", B=32, new_lo=1, new_hi=1, ctx_lo=100,
             ctx_hi=4000, Hkv=8, ps=64, block=16, codes="e4m3", layout="HND", dtype="bf16",
             mix=11),
        # prompt chunks of ragged lengths, a scale for each token
        dict(name="store8_chunk_i8", op="store", B=12, new_lo=400, new_hi=2400, ctx_lo=0,
             ctx_hi=3000, Hkv=8, ps=16, block=1, codes="i8", layout="NHD", dtype="f16", mix=12),
        # four short prefixes back to 16 bits
        dict(name="load8_short", op="load", B=4, new_lo=0, new_hi=0, ctx_lo=60, ctx_hi=500, Hkv=8,
             ps=16, block=16, codes="i8", layout="NHD", dtype="f16", mix=13),
        # eight long ones
        dict(name="load8_long", op="load", B=8, new_lo=0, new_hi=0, ctx_lo=2000, ctx_hi=16000,
             Hkv=8, ps=64, block=64, codes="e4m3", layout="HND", dtype="bf16", mix=14),
        # a single user's decode step at a short context: latency
        dict(name="paged8_decode_one", op="paged", B=1, Hq=32, Hkv=8, ps=16, block=1,
             codes="i8", layout="NHD", dtype="f16", ctx_lo=1000, ctx_hi=1000, new_lo=1, new_hi=1,
             chunk=0, kind="causal", window=0, first=0, sink=False, mix=15),
        # a batch of decodes at ragged contexts: the cache's bandwidth
        dict(name="paged8_decode_b64", op="paged", B=64, Hq=64, Hkv=8, ps=64, block=16,
             codes="e4m3", layout="HND", dtype="bf16", ctx_lo=2000, ctx_hi=16000, new_lo=1,
             new_hi=1, chunk=0, kind="causal", window=0, first=0, sink=True, mix=16),
        # two users at long contexts, a few speculated tokens each
        dict(name="paged8_decode_long", op="paged", B=2, Hq=32, Hkv=4, ps=32, block=32,
             codes="i8", layout="HND", dtype="bf16", ctx_lo=60000, ctx_hi=130000, new_lo=3,
             new_hi=5, chunk=0, kind="causal", window=0, first=0, sink=False, mix=17),
        # chunks of two prompts over what is cached already: the tensor cores
        dict(name="paged8_chunk_b2", op="paged", B=2, Hq=32, Hkv=8, ps=64, block=64,
             codes="e4m3", layout="HND", dtype="bf16", ctx_lo=7000, ctx_hi=9001, new_lo=1800,
             new_hi=2048, chunk=0, kind="causal", window=0, first=0, sink=False, mix=18),
        # a step of a model with a window and first tokens: decodes beside one chunk
        dict(name="paged8_window_mixed", op="paged", B=16, Hq=32, Hkv=8, ps=32, block=1,
             codes="e4m3", layout="NHD", dtype="f16", ctx_lo=500, ctx_hi=16000, new_lo=1,
             new_hi=4, chunk=500, kind="first", window=1024, first=4, sink=True, mix=19),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "store", "load", "paged", "paged"])
    dtype = rng.choice(["f16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        return dict(op=op, back=rng.random() < 0.5, layout=rng.choice(["rows", "heads"]),
                    B=rng.choice([1, 1, 2, 3]), S=_log(rng, 1, 5000), Hq=Hkv * group, Hkv=Hkv,
                    dtype=dtype, rot=16 * rng.randint(1, 8), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0]),
                    scaling=rng.choice(["none", "linear", "raised", "parts"]),
                    far=_log(rng, 10, 1 << 22))
    ps = rng.choice([16, 32, 48, 64, 128])
    block = rng.choice([b for b in (1, 16, 32, 64) if ps % b == 0])
    case = dict(op=op, Hkv=Hkv, ps=ps, block=block, codes=rng.choice(["e4m3", "i8"]),
                layout=rng.choice(["HND", "NHD"]), dtype=dtype, mix=rng.randrange(1 << 30))
    if op == "store":
        new, B = _log(rng, 1, 1500), _log(rng, 1, 16)
        return dict(case, B=B, new_lo=1, new_hi=new, ctx_lo=0, ctx_hi=_log(rng, 1, 3000))
    if op == "load":
        return dict(case, B=_log(rng, 1, 12), new_lo=0, new_hi=0, ctx_lo=1,
                    ctx_hi=_log(rng, 1, 8000))
    kind = rng.choice(["causal", "first", "first", "sliding"])
    # decode steps, speculated tokens, chunks: the longer the chunk the fewer requests
    new = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 8, 1000)])
    return dict(case, B=_log(rng, 1, 48 if new <= 8 else 6), Hq=Hkv * group, ctx_lo=1,
                ctx_hi=_log(rng, 64, 16000 if new <= 8 else 6000), new_lo=1, new_hi=new, chunk=0,
                kind=kind, window=_log(rng, 1, 4096) if kind != "causal" else 0,
                first=_log(rng, 1, 300) if kind == "first" else 0, sink=rng.random() < 0.5)


def _lengths(case):
    """(new tokens, earlier tokens) of each request; for `paged` (new tokens,
    keys).  They belong to the case, so that its work is known without its
    inputs."""
    r = random.Random(case["mix"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    if case.get("chunk"):
        new[r.randrange(case["B"])] = case["chunk"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in new]
    return new, ([max(n, c) for n, c in zip(new, ctx)] if case["op"] == "paged" else ctx)


def _spans(case):
    """What `store` and `load` read back: (first position, rows) of each request,
    from the first row of the block that the new tokens begin in."""
    new, old = _lengths(case)
    if case["op"] == "load":
        return [(0, c) for c in old]
    first = [c // case["block"] * case["block"] for c in old]
    return [(f, c + n - f) for n, c, f in zip(new, old, first)]


def _rule(case):
    """(window, first) of the causal rule: key j is visible to position i when
    j <= i and (i - j < window or j < first)."""
    return (case["window"] or 1 << 30), case["first"]


def _frequencies(case):
    """Radians a position of each pair, and what cos and sin are multiplied by."""
    R, base = case["rot"], case["base"]
    if case["scaling"] == "raised":    # twice the context by a larger base
        base *= 2.0 ** (R / (R - 2.0))
    w = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if case["scaling"] == "linear":
        return [x / 4.0 for x in w], 1.0
    if case["scaling"] != "parts":
        return w, 1.0
    # eight times a context of 4096: pairs that turn more than 32 times in it keep
    # their rate, those that turn less than once take an eighth
    out = []
    for x in w:
        turns = 4096 * x / (2.0 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
        out.append(x * (keep + (1.0 - keep) / 8.0))
    return out, 0.1 * math.log(8.0) + 1.0


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rope_handle(case):
    from masked_attention_backward_gb300 import binding as mab
    scaling = {"none": None, "linear": mab.RopeScaling("linear", 4.0),
               "raised": mab.RopeScaling("raised", 2.0),
               "parts": mab.RopeScaling("parts", 8.0, original_length=4096)}[case["scaling"]]
    return mab.Rope(case["rot"], base=case["base"], interleaved=case["interleaved"],
                    scaling=scaling, device="cuda")


def _pages(case, g, P):
    """A cache of P pages with codes and scales as earlier tokens left them."""
    Hkv, ps, block = case["Hkv"], case["ps"], case["block"]
    shape = (P, Hkv, ps, D) if case["layout"] == "HND" else (P, ps, Hkv, D)
    out = []
    for _ in range(2):
        pages = torch.empty(shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(P, Hkv, ps // block, dtype=torch.uint8, device="cuda")
        for lo in range(0, P, 512):  # a part at a time: 32-bit values take four times the room
            hi = min(lo + 512, P)
            x = torch.randn((hi - lo, Hkv, ps // block, block, D), generator=g, device="cuda")
            # blocks of different magnitude, as channels and tokens have
            x *= torch.exp2(torch.randint(-2, 2, x.shape[:3], generator=g,
                                          device="cuda").float())[..., None, None]
            e = _exponent(case, x.abs().amax((-1, -2)))
            c = _round(case, x * _two(-e)[..., None, None], e[..., None, None])
            c = c.reshape(hi - lo, Hkv, ps, D)
            pages[lo:hi] = c if case["layout"] == "HND" else c.transpose(1, 2)
            s[lo:hi] = (e + 127).to(torch.uint8)
        out += [pages, s]
    return out[0].view(CODES[case["codes"]]), out[2].view(CODES[case["codes"]]), out[1], out[3]


def _table(case, g, held, spare):
    P = sum(held) + spare
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    h = _ints(held).long()
    col = torch.arange(max(held) + 1, device="cuda")[None, :]
    start = h.cumsum(0) - h
    return torch.where(col < h[:, None], perm[(start[:, None] + col).clamp(max=P - 1)],
                       torch.full_like(perm[:1], -1)), P


def _offsets(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return _ints(out)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    dt = DTYPES[case["dtype"]]
    Hkv = case["Hkv"]
    if op == "rope":
        B, S, Hq = case["B"], case["S"], case["Hq"]
        if case["layout"] == "rows":   # slices of a fused projection's output
            qkv = _normal(g, (B * S, Hq + 2 * Hkv, D), dt)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            st["q"], st["k"] = _normal(g, (B, Hq, S, D), dt), _normal(g, (B, Hkv, S, D), dt)
        if case["far"]:
            n = (B * S,) if case["layout"] == "rows" else (B, S)
            st["position"] = torch.randint(0, case["far"], n, generator=g, device="cuda",
                                           dtype=torch.int32)
        else:
            st["position"] = None
        w, st["factor"] = _frequencies(case)
        st["w"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        if own:
            st["rope"] = _rope_handle(case)
        return st
    ps = case["ps"]
    if op == "paged":
        new, ctx = _lengths(case)
        st["block_table"], P = _table(case, g, [-(-n // ps) for n in ctx], 7)
        Hq, T = case["Hq"], sum(new)
        st["q"] = _normal(g, (T, Hq, D), dt)
        st["sink"] = torch.randn(Hq, generator=g, device="cuda") if case["sink"] else None
        st.update(cu=_offsets(new), seqlen_k=_ints(ctx), T=T, max_q=max(new), max_k=max(ctx),
                  scale=1.0 / math.sqrt(D))
    else:
        new, old = _lengths(case)
        st["block_table"], P = _table(case, g, [-(-(n + c) // ps) for n, c in zip(new, old)], 5)
        spans = _spans(case)
        n = [r for _, r in spans]
        st.update(start=_ints([f for f, _ in spans]), cu_back=_offsets(n), T_back=sum(n))
        if op == "store":
            T = sum(new)
            qkv = _normal(g, (T, 3 * Hkv, D), dt)   # slices of a fused projection's output
            st["k"], st["v"] = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
            cu = _offsets(new).long()
            t = torch.arange(T, device="cuda")
            b = torch.searchsorted(cu[1:], t, right=True)
            pos = _ints(old).long()[b] + t - cu[b]
            st["slot_map"] = st["block_table"][b, pos // ps].long() * ps + pos % ps
    st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"] = _pages(case, g, P)
    return st


# ------------------------------------------------------------------ plain forms

def _two(e):
    """2^e for whole numbers e, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(case, amax):
    """The least e with amax <= top * 2^e, as float32."""
    m, x = torch.frexp(amax)                   # amax = m 2^x, m in [0.5, 1)
    tm, tx = math.frexp(TOP[case["codes"]])
    e = x - tx + (m > tm).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -1000))
    return e.clamp(min=LEAST[case["codes"], case["dtype"]]).float()


def _round(case, x, e):
    """Codes (their bytes) of values x in units of 2^e; the value of a code stays
    finite in the cache's 16-bit type."""
    big = {("e4m3", "f16"): 8, ("i8", "f16"): 10, ("e4m3", "bf16"): 120,
           ("i8", "bf16"): 122}[case["codes"], case["dtype"]]
    lim = torch.where(e >= big, 240.0 if case["codes"] == "e4m3" else 63.0, TOP[case["codes"]])
    if case["codes"] == "i8":
        x = torch.round(x)
    x = torch.maximum(torch.minimum(x, lim), -lim)
    return x.to(CODES[case["codes"]]).view(torch.uint8)


def _plain_rope(st):
    case = st["case"]
    R, h = case["rot"], case["rot"] // 2
    pos = st["position"]
    if pos is None:
        pos = torch.arange(case["S"], device="cuda")
    angle = pos[..., None].double() * st["w"]
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()
    if case["back"]:
        sin = -sin
    if case["layout"] == "rows":   # [T, 1, h]
        cos, sin = cos[:, None], sin[:, None]
    elif cos.dim() == 3:           # [B, 1, S, h]
        cos, sin = cos[:, None], sin[:, None]
    out = []
    for x in (st["q"], st["k"]):
        y = x.float()
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["interleaved"] else (y[..., :h], y[..., h:R])
        p, q = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([p, q], -1).flatten(-2) if case["interleaved"] else \
            torch.cat([p, q], -1)
        out.append(torch.cat([turned, y[..., R:]], -1).to(x.dtype))
    return tuple(out)


def _rows_first(case, pages):
    """Pages as [P, blocks, block, Hkv, D]: a view."""
    x = pages.view(torch.uint8) if pages.dtype != torch.uint8 else pages
    x = x.transpose(1, 2) if case["layout"] == "HND" else x
    return x.unflatten(1, (case["ps"] // case["block"], case["block"]))


def _plain_store(st):
    case = st["case"]
    ps, block = case["ps"], case["block"]
    slot = st["slot_map"]
    per = ps // block
    blk, row = slot // block, slot % block
    ids, which = torch.unique(blk, return_inverse=True)
    start = torch.full_like(ids, block).scatter_reduce_(0, which, row, "amin")
    for pages, scales, x in ((st["k_pages"], st["k_scales"], st["k"]),
                             (st["v_pages"], st["v_scales"], st["v"])):
        x = x.float()
        need = torch.full((ids.numel(), case["Hkv"]), -1000.0, device="cuda")
        need.scatter_reduce_(0, which[:, None].expand(-1, case["Hkv"]),
                             _exponent(case, x.abs().amax(-1)), "amax")
        had = scales[ids // per, :, ids % per].float() - 127
        e = torch.where(start[:, None] > 0, torch.maximum(need, had), need)
        codes = _rows_first(case, pages)
        rows = codes[ids // per, ids % per]                  # [n, block, Hkv, D]
        vals = rows.view(CODES[case["codes"]]).float() * _two(had - e)[:, None, :, None]
        again = _round(case, vals, e[:, None, :, None])
        live = torch.arange(block, device="cuda")[None, :] < start[:, None]
        rows = torch.where(live[..., None, None], again, rows)
        ex = e[which][..., None]
        rows[which, row] = _round(case, x * _two(-ex), ex)
        codes[ids // per, ids % per] = rows
        scales[ids // per, :, ids % per] = (e + 127).to(torch.uint8)
    return _plain_load(st) + (st["k_scales"], st["v_scales"])


def _plain_load(st):
    case = st["case"]
    ps, block = case["ps"], case["block"]
    cu = st["cu_back"].long()
    t = torch.arange(st["T_back"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = st["start"].long()[b] + t - cu[b]
    page = st["block_table"][b, pos // ps].long()
    at = (pos % ps) // block
    out = []
    for pages, scales in ((st["k_pages"], st["k_scales"]), (st["v_pages"], st["v_scales"])):
        c = _rows_first(case, pages)[page, at, pos % block].view(CODES[case["codes"]]).float()
        s = _two(scales[page, :, at].int() - 127)
        out.append((c * s[..., None]).to(DTYPES[case["dtype"]]))
    return tuple(out)


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
    ps, block, (window, first) = case["ps"], case["block"], _rule(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    g, B = Hq // Hkv, case["B"]
    table = st["block_table"][:, :-(-st["max_k"] // ps)].long().clamp(min=0)
    Lp = table.shape[1] * ps

    def rows(pages, scales):  # [B, Hkv, 1, Lp, D]
        c = _rows_first(case, pages)[table].view(CODES[case["codes"]])
        s = _two(scales[table].int() - 127)   # [B, cols, Hkv, blocks]
        x = c.float() * s.transpose(2, 3)[:, :, :, None, :, None]
        return x.reshape(B, Lp, Hkv, D).permute(0, 2, 1, 3).unsqueeze(2)

    cu, L = st["cu"].long(), st["seqlen_k"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(st["max_q"], device="cuda")
    tok = (cu[:-1, None] + i).clamp(max=st["T"] - 1)
    q = st["q"][tok].float().reshape(B, -1, Hkv, g, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q, rows(st["k_pages"], st["k_scales"]).transpose(-1, -2)) * st["scale"]
    pos = (L - n)[:, None, None] + i[None, :, None]
    j = torch.arange(Lp, device="cuda")[None, None, :]
    vis = (j <= pos) & (j < L[:, None, None]) & ((pos - j < window) | (j < first))
    s = torch.where(vis[:, None, None], s, NEG)
    sink = None if st["sink"] is None else st["sink"].reshape(Hkv, g, 1, 1)
    o, lse = _softmax(s, sink, rows(st["v_pages"], st["v_scales"]))
    # back to the packed rows of the new tokens
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, D)[b, t - cu[b]]
    lse = lse.permute(0, 3, 1, 2).reshape(B, -1, Hq)[b, t - cu[b]]
    return o.to(st["q"].dtype), lse.t().contiguous()


# ------------------------------------------------------------------ one pass

def _own_run(st):
    from masked_attention_backward_gb300 import binding as mab
    case = st["case"]
    op = case["op"]
    if op == "rope":
        if "rope" not in st:
            st["rope"] = _rope_handle(case)
        turn = mab.rope_bwd if case["back"] else mab.rope
        return turn(st["rope"], st["q"], st["k"], st["position"])
    cache = mab.PagedCache8(st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"],
                            DTYPES[case["dtype"]], case["layout"])
    if op == "paged":
        kind = {"causal": mab.ATTN_MASK_CAUSAL, "sliding": mab.ATTN_MASK_SLIDING,
                "first": mab.ATTN_MASK_SLIDING_FIRST}[case["kind"]]
        mask = mab.Mask(kind=kind, window=case["window"], first=case["first"],
                        cu_seqlens_q=st["cu"], seqlen_k=st["seqlen_k"], max_seqlen_q=st["max_q"],
                        max_seqlen_k=st["max_k"], total_q=st["T"])
        return mab.paged_fwd(st["q"], cache, st["block_table"], st["sink"], mask, st["scale"])
    if op == "store":
        mab.paged_store(cache, st["k"], st["v"], st["slot_map"])
    k, v = mab.paged_load(cache, st["block_table"], st["cu_back"], st["T_back"], st["start"])
    return (k, v, st["k_scales"], st["v_scales"]) if op == "store" else (k, v)


def run(st):
    if own:
        return _own_run(st)
    return {"rope": _plain_rope, "store": _plain_store, "load": _plain_load,
            "paged": _plain_paged}[st["case"]["op"]](st)


# ------------------------------------------------------------------ the work

def _pairs(positions, window, first):
    pos = np.asarray(positions, dtype=np.int64)
    return int((np.minimum(pos + 1, window) +
                np.clip(np.minimum(pos - window + 1, first), 0, None)).sum())


def work(case):
    op, Hkv = case["op"], case["Hkv"]
    if op == "rope":
        rows = case["B"] * case["S"] * (case["Hq"] + Hkv)
        pos = 4 * case["B"] * case["S"] if case["far"] else 0
        return {"bytes": rows * D * 2 * 2 + pos, "flops": rows * case["rot"] * 3}
    row8 = Hkv * D + Hkv / case["block"]   # codes and scales of a token, K or V
    if op in ("store", "load"):
        new, _ = _lengths(case)
        back, T = sum(n for _, n in _spans(case)), sum(new)
        moved = back * 2 * (row8 + Hkv * D * 2)                    # read back to 16 bits
        if op == "store":
            moved += T * (8 + 2 * (Hkv * D * 2 + row8)) + (back - T) * 2 * row8
        return {"bytes": int(moved), "flops": 0}
    window, first = _rule(case)
    Hq = case["Hq"]
    new, ctx = _lengths(case)
    pairs = keys = 0
    for n, L in zip(new, ctx):
        pairs += _pairs(np.arange(L - n, L), window, first)
        lo = max(0, L - n - window + 1)
        keys += L - lo + min(first, lo)
    T = sum(new)
    return {"bytes": int(2 * T * Hq * D * 2 + T * Hq * 4 + 2 * keys * row8),
            "flops": 4 * D * pairs * Hq}


# ------------------------------------------------------------------ 64 bits

def _two64(e):
    """2^e for whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values64(case, pages, scales, ids):
    """Rows of the pages `ids` in order, [n * ps, Hkv, D] in 64 bits."""
    c = pages[ids] if case["codes"] == "i8" else \
        pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    c = c.double()
    c = c.transpose(1, 2) if case["layout"] == "HND" else c        # [n, ps, Hkv, D]
    s = _two64(scales[ids].int() - 127)
    return (c * s.transpose(1, 2).repeat_interleave(case["block"], 1)[..., None]).flatten(0, 1)


def _nearest64(case, x, e):
    """x to the nearest value of a code times 2^e (ties to even), in 64 bits."""
    unit = _two64(e)
    y = x / unit
    limit = {"f16": 65504.0, "bf16": (2 - 2.0 ** -7) * 2.0 ** 127}[case["dtype"]]
    if case["codes"] == "i8":
        y = torch.round(y).clamp(-127, 127)
        over = torch.floor(limit / unit)
        return torch.minimum(torch.maximum(y, -over), over) * unit
    step = _two64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    y = (torch.round(y / step) * step).clamp(-448, 448)
    y = torch.where(y.abs() * unit > limit, torch.sign(y) * 240, y)
    return y * unit


def _exact_store(case, st):
    """One request after another; what is read back, and the scales."""
    ps, block, Hkv = case["ps"], case["block"], case["Hkv"]
    new, old = _lengths(case)
    least, top = LEAST[case["codes"], case["dtype"]], TOP[case["codes"]]
    out = []
    for pages, scales, x in ((st["k_pages"], st["k_scales"], st["k"]),
                             (st["v_pages"], st["v_scales"], st["v"])):
        scales, got, t0 = scales.clone(), [], 0
        for b, (n, c) in enumerate(zip(new, old)):
            lo, hi = c // block, -(-(c + n) // block)         # the blocks that are written
            ids = st["block_table"][b, :-(-(c + n) // ps)].long()
            vals = _values64(case, pages, scales, ids)[:hi * block]
            vals = torch.cat([vals, vals.new_zeros(hi * block - vals.shape[0], Hkv, D)])
            rows = vals[lo * block:].clone()
            head = c - lo * block                             # rows that were there
            rows[head:] = 0
            rows[head:head + n] = x[t0:t0 + n].double()
            t0 += n
            blocks = rows.unflatten(0, (hi - lo, block))
            fresh = blocks.clone()
            fresh[0, :head] = 0
            amax = fresh.abs().amax((1, 3))                   # [blocks, Hkv]
            e = torch.ceil(torch.log2((amax / top).clamp(min=2.0 ** -200))).int()
            e = torch.where(amax > top * _two64(e), e + 1, e)
            e = torch.where(amax <= top * _two64(e - 1), e - 1, e).clamp(min=least)
            at = torch.arange(lo, hi, device="cuda")
            page, col = ids[at * block // ps], at % (ps // block)
            if head:
                e[0] = torch.maximum(e[0], scales[page[0], :, col[0]].int() - 127)
            scales[page, :, col] = (e + 127).to(torch.uint8)
            back = _nearest64(case, blocks, e[:, None, :, None])
            got.append(back.flatten(0, 1)[:head + n])
        out.append((torch.cat(got), scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _attend64(q, k, v, vis, sink, scale):
    """One head: rows q [n, D] over keys k, values v [l, D] under vis [n, l]."""
    s = (q.double() @ k.T * scale).masked_fill(~vis, NEG)
    if sink is not None:
        s = torch.cat([s, sink.double().expand(s.shape[0], 1)], 1)
    lse = torch.logsumexp(s, 1)
    seen = lse > NEG
    p = torch.exp(s - torch.where(seen, lse, 0.0)[:, None])[:, :k.shape[0]]
    return p @ v, torch.where(seen, lse, math.inf)


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "rope":
        R, (w, factor) = case["rot"], _frequencies(case)
        rows = case["layout"] == "rows"
        pos = st["position"]
        pos = torch.arange(case["S"], device="cuda") if pos is None else pos
        out = []
        for x in (st["q"], st["k"]):
            y = x.double().clone()
            for i, wi in enumerate(w):
                a = pos.double() * wi
                a = a[:, None] if rows else a[:, None, :] if a.dim() == 2 else a
                turn = torch.polar(torch.full_like(a, factor), -a if case["back"] else a)
                d0, d1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
                z = torch.complex(y[..., d0], y[..., d1]) * turn
                y[..., d0], y[..., d1] = z.real, z.imag
            out.append(y)
        return tuple(out)
    if op == "store":
        return _exact_store(case, st)
    ps = case["ps"]
    if op == "load":
        out = [[], []]
        for b, (first, n) in enumerate(_spans(case)):
            ids = st["block_table"][b, :-(-(first + n) // ps)].long()
            for o, x in zip(out, "kv"):
                o.append(_values64(case, st[x + "_pages"], st[x + "_scales"],
                                   ids)[first:first + n])
        return torch.cat(out[0]), torch.cat(out[1])
    window, first = _rule(case)
    Hq, group = case["Hq"], case["Hq"] // case["Hkv"]
    new, ctx = _lengths(case)
    o = torch.zeros(st["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(Hq, st["T"], dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, L) in enumerate(zip(new, ctx)):
        ids = st["block_table"][b, :-(-L // ps)].long()
        ks = _values64(case, st["k_pages"], st["k_scales"], ids)[:L]
        vs = _values64(case, st["v_pages"], st["v_scales"], ids)[:L]
        i = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        vis = (i >= j) & ((j > i - window) | (j < first))
        for h in range(Hq):
            o[t0:t0 + n, h], lse[h, t0:t0 + n] = _attend64(
                st["q"][t0:t0 + n, h], ks[:, h // group], vs[:, h // group], vis,
                None if st["sink"] is None else st["sink"][h], st["scale"])
        t0 += n
    return o, lse
