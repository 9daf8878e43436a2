"""Attention over the 8-bit cache against plain 64-bit attention over the values
that its codes and scales stand for, one request and head at a time, within
attn64's bounds (the values are exact in 16 bits, so no rounding joins those of the
16-bit cache).  Unless a test says otherwise, rows and blocks that no new token
sees hold codes without a number and scales of NaN, and the table holds -7 where no
key of a page is seen."""
import math
import random

import pytest
import torch

import attn64
import quant64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SCALE = 1.0 / math.sqrt(128)
NONE, CAUSAL, SLIDING, FIRST = (mab.ATTN_MASK_NONE, mab.ATTN_MASK_CAUSAL, mab.ATTN_MASK_SLIDING,
                                mab.ATTN_MASK_SLIDING_FIRST)
FORMS = [("e4m3", F16), ("e4m3", BF16), ("i8", F16), ("i8", BF16)]
IDS = ["e4m3-f16", "e4m3-bf16", "i8-f16", "i8-bf16"]


@pytest.fixture(autouse=True)
def _use_room(monkeypatch):
    """Chunks of any size use room in the workspace."""
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")


class Case:
    """reqs: (new tokens, keys) of each request."""

    def __init__(self, reqs, Hq=4, Hkv=2, ps=16, block=16, form=("e4m3", BF16), layout="HND",
                 kind=CAUSAL, window=0, first=0, sink=True, seed=0, pad=0, spare_cols=1,
                 spread=3):
        g = torch.Generator("cpu").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        code, dtype = form
        self.reqs, self.kind, self.window, self.first = reqs, kind, window, first
        self.Hq, self.Hkv, self.ps, self.dtype = Hq, Hkv, ps, dtype
        held = [-(-L // ps) for _, L in reqs]
        P, cols = sum(held) + 3, max(held) + spare_cols
        ids = list(range(P))
        random.Random(seed).shuffle(ids)
        table = torch.full((len(reqs), cols), -7, dtype=torch.int32)
        self.vis, live = [], torch.zeros(P, ps, dtype=torch.bool)
        at, rows = 0, []
        for b, (n, L) in enumerate(reqs):
            x, j = torch.arange(L - n, L), torch.arange(L)
            vis = attn64.window_first(x, j, None if kind == CAUSAL else window,
                                      first if kind == FIRST else 0)
            if kind == NONE:
                vis = torch.ones(n, L, dtype=torch.bool)
            seen = vis.any(0)
            pages = torch.tensor(ids[at:at + held[b]], dtype=torch.long)
            at += held[b]
            rows.append(pages[j // ps] * ps + j % ps if L else torch.zeros(0, dtype=torch.long))
            live.view(-1)[rows[b][seen]] = True
            for c in range(held[b]):
                if bool(seen[c * ps:(c + 1) * ps].any()):
                    table[b, c] = int(pages[c])
            self.vis.append(vis.cuda())
        caches = []
        per = ps // block
        for _ in range(2):
            # each block at a magnitude of its own, its exponent up to two larger than
            # need be (as one that joined larger rows has it)
            c = quant64.Cache64(P, Hkv, ps, block, code, dtype)
            m = torch.randint(-spread, spread + 1, (P, Hkv, per), generator=g)
            top = math.frexp(quant64.TOP[code])[1]
            c.exp = m + 3 - top + torch.randint(0, 3, m.shape, generator=g)
            x = r(P, ps, Hkv, 128).double() * \
                torch.exp2(m.double()).repeat_interleave(block, 2).transpose(1, 2)[..., None]
            unit = torch.exp2(c.exp.double()).repeat_interleave(block, 2).transpose(1, 2)[..., None]
            c.num = quant64.nearest(code, x / unit, quant64.TOP[code])
            caches.append(c)
        vals = [c.values(torch.arange(P * ps)) for c in caches]
        self.k = [vals[0][s].cuda() for s in rows]
        self.v = [vals[1][s].cuda() for s in rows]
        self.cache = quant64.make(*caches, layout)
        # what nobody sees
        dead = ~live
        junk = 0x7f if code == "e4m3" else 0x80
        d = dead[:, None, :, None] if layout == "HND" else dead[:, :, None, None]
        for c in (self.cache.k_pages, self.cache.v_pages):
            u = c.view(torch.uint8)
            u.copy_(torch.where(d.cuda(), torch.full_like(u, junk), u))
        gone = dead.view(P, 1, per, block).all(3).expand(P, Hkv, per).cuda()
        for s in (self.cache.k_scales, self.cache.v_scales):
            s.copy_(torch.where(gone, torch.full_like(s, 255), s))
        self.table = table.cuda()
        self.T = sum(n for n, _ in reqs) + pad
        self.q = r(self.T, Hq, 128).to(dtype).cuda()
        self.sink = r(Hq).cuda() if sink else None
        cu = [0]
        for n, _ in reqs:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor([L for _, L in reqs], dtype=torch.int32, device="cuda")
        self.mask = mab.Mask(kind=kind, window=window, first=first, cu_seqlens_q=self.cu,
                             seqlen_k=self.lens, total_q=self.T,
                             max_seqlen_q=max(max(n for n, _ in reqs), 1),
                             max_seqlen_k=max(max(L for _, L in reqs), 1))

    def workspace(self, room=True):
        """With room for the chunks' rows in 16 bits, or the least."""
        shape = mab.paged_shape(self.q, self.cache, self.mask)
        n = mab.attn_paged8_workspace_size(shape, self.mask.desc() if room else None)[1]
        return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")

    def run(self, room=True, **kw):
        ws = self.workspace(room)
        out = (torch.full_like(self.q, 7.0),
               torch.full((self.Hq, self.T), 7.0, device="cuda"))
        mab.paged_fwd(self.q, self.cache, self.table, self.sink, self.mask, SCALE, ws=ws, out=out,
                      **kw)
        torch.cuda.synchronize()
        return out, mab.device_status(ws)

    def check(self, o, lse):
        g, t0 = self.Hq // self.Hkv, 0
        for b, (n, L) in enumerate(self.reqs):
            for h in range(self.Hq):
                ro, rl, ob, lb = attn64.head_fwd(
                    self.q[t0:t0 + n, h], self.k[b][:, h // g], self.v[b][:, h // g], self.vis[b],
                    None if self.sink is None else float(self.sink[h]), SCALE)
                attn64.check(f"o of request {b} head {h}", o[t0:t0 + n, h], ro, ob)
                attn64.check(f"lse of request {b} head {h}", lse[h, t0:t0 + n], rl, lb)
            t0 += n
        # rows behind the last request stay as they were
        assert bool((o[t0:] == 7).all()) and bool((lse[:, t0:] == 7).all())


def _go(*a, room=True, **kw):
    c = Case(*a, **kw)
    (o, lse), status = c.run(room)
    assert status == mab.ATTN_OK
    c.check(o, lse)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 640, 1001])
def test_one_token(cuda_lib, L, form):
    _go([(1, L)], form=form, block=1 if L % 3 else 16, sink=L % 2 == 0, seed=L)


@pytest.mark.parametrize("n,L", [(1, 1), (2, 2), (3, 70), (64, 64), (65, 65), (127, 300),
                                 (200, 1000), (500, 500)])
@pytest.mark.parametrize("kind,window,first", [(CAUSAL, 0, 0), (SLIDING, 1, 0), (SLIDING, 70, 0),
                                               (FIRST, 40, 3), (FIRST, 100, 130), (NONE, 0, 0)])
@pytest.mark.parametrize("room", [True, False])
def test_chunks(cuda_lib, n, L, kind, window, first, room):
    _go([(n, L)], room=room, kind=kind, window=window, first=first, seed=n + L, pad=3,
        block=1 if n % 2 else 16, form=FORMS[(n + window) % 4])


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("ps,block", [(16, 1), (16, 16), (32, 32), (48, 1), (48, 16), (64, 64),
                                      (80, 16), (128, 32), (128, 64), (256, 1)])
@pytest.mark.parametrize("room", [True, False])
def test_pages(cuda_lib, ps, block, layout, room):
    _go([(1, 700), (5, 333), (90, 91)], room=room, ps=ps, block=block, layout=layout, seed=ps,
        form=FORMS[ps // 16 % 4])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 1), (9, 1), (16, 2), (33, 1),
                                    (64, 8), (128, 1)])
@pytest.mark.parametrize("n", [1, 2, 4, 17])
@pytest.mark.parametrize("room", [True, False])
def test_heads(cuda_lib, Hq, Hkv, n, room):
    _go([(n, 150), (1, 30)], room=room, Hq=Hq, Hkv=Hkv, seed=Hq + n, form=FORMS[n % 4], block=16)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("new", [1, 4])
def test_long_context_over_many_ctas(cuda_lib, form, new):
    _go([(new, 20011)], Hq=8, Hkv=2, ps=64, block=64 if new == 1 else 1, form=form, seed=new)


@pytest.mark.parametrize("kind,window,first", [(CAUSAL, 0, 0), (FIRST, 200, 5)])
@pytest.mark.parametrize("room", [True, False])
def test_ragged_batch(cuda_lib, kind, window, first, room):
    """Requests without new tokens, without keys, single tokens, chunks."""
    r = random.Random(7)
    reqs = [(1, r.randint(1, 900)) for _ in range(12)]
    reqs += [(0, 50), (0, 0), (130, 700), (3, 3), (1, 1), (9, 2000), (0, 0), (2, 511)]
    r.shuffle(reqs)
    _go(reqs, room=room, Hq=8, Hkv=2, ps=32, block=16, kind=kind, window=window, first=first,
        pad=5, seed=3)


@pytest.mark.parametrize("room", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (20, 1), (6, 2)])
def test_few_rows_beside_chunks(cuda_lib, Hq, Hkv, room):
    """Requests on both sides of the number of rows that makes a chunk."""
    g = Hq // Hkv
    few = 16 // g
    reqs = [(max(few, 1), 100), (few + 1, 333), (1, 64), (130, 131), (0, 9), (0, 0), (few + 2, 65),
            (max(few - 1, 1), 2000), (200, 777)]
    _go(reqs, room=room, Hq=Hq, Hkv=Hkv, ps=16, block=16, kind=FIRST, window=90, first=20, pad=2)
    _go(reqs, room=room, Hq=Hq, Hkv=Hkv, ps=64, block=1, form=("i8", F16))


def test_workspace(monkeypatch):
    """The least need does not grow with the lengths; the room goes by what chunks see."""
    shape = lambda **kw: mab.attn_shape_t(*[dict(dict(B=2, Hq=8, Hkv=2, Sq=1, Skv=6400, D=128,
                                                      dtype=0, flags=0), **kw)[n]
                                            for n in ("B", "Hq", "Hkv", "Sq", "Skv", "D", "dtype",
                                                      "flags")])
    least = lambda s: mab.attn_paged8_workspace_size(s)[1]
    mask = lambda **kw: mab.attn_mask_desc_t(kind=CAUSAL, **kw)
    full = lambda s, **kw: mab.attn_paged8_workspace_size(s, mask(**kw))[1]
    assert least(shape(Sq=128)) == least(shape(Sq=4000, Skv=2 ** 24))
    assert full(shape(), total_q=2) == least(shape())
    assert full(shape(Sq=32), total_q=64) == least(shape(Sq=32))   # one tile a kv head
    s = shape(Sq=500)
    page = 2 * 2 * 64 * 128 * 2                                    # K and V of both heads
    one = full(s, total_q=9) - least(s)                            # room for one chunk
    assert 100 * page <= one < 101 * page
    assert 200 * page <= full(s, total_q=1000) - least(s) < 201 * page
    m = mab.attn_mask_desc_t(kind=FIRST, window=640, first=64, total_q=500)
    seen = mab.attn_paged8_workspace_size(s, m)[1] - least(s)
    assert 2 * 20 * page <= seen < 2 * 24 * page
    # without the hook: where the bounds promise 40 steps an SM, of
    # ceil(total_q * 4 / 128) * 100 * 2 / 152
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM")
    assert full(s, total_q=960) == least(s) and full(s, total_q=1000) > least(s)
    assert mab.attn_paged8_workspace_size(shape(D=64), mask())[0] == mab.ATTN_ERR_UNSUPPORTED
    assert mab.attn_paged8_workspace_size(shape(B=0))[0] == mab.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_more_new_tokens_than_keys(cuda_lib, form):
    """Rows before position zero see nothing: the sink, or +inf."""
    for sink in (True, False):
        c = Case([(1, 40), (1, 8)], form=form, sink=sink)
        # request 0 brings one token over no key at all
        c.lens[0] = 0
        c.reqs[0] = (1, 0)
        c.vis[0], c.k[0], c.v[0] = c.vis[0][:, :0], c.k[0][:0], c.v[0][:0]
        (o, lse), status = c.run()
        assert status == mab.ATTN_OK
        c.check(o, lse)


@pytest.mark.parametrize("n", [1, 30, 90])
@pytest.mark.parametrize("room", [True, False])
@pytest.mark.parametrize("other", [0, 1, 100])
def test_bad_page(cuda_lib, n, room, other):
    """A page outside the cache stands for zeros, and the status says so, whichever
    kernel meets it."""
    c = Case([(n, 100), (other, 200)], ps=16, block=1, form=("i8", F16))
    for bad in (c.cache.num_pages, -1, -2 ** 31, 2 ** 31 - 1):
        c.table[0, 2] = bad
        c.k[0][32:48] = 0
        c.v[0][32:48] = 0
        (o, lse), status = c.run(room)
        assert status == mab.ATTN_ERR_INVALID_ARG
        c.check(o, lse)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [1, 20])
def test_extreme_scales(cuda_lib, form, n):
    """Exponents over the whole range that the store gives values of size 2^-12
    to 2^12, beside each other."""
    _go([(n, 300)], form=form, block=16, spread=6, seed=5)
    _go([(n, 300)], form=form, block=1, spread=6, seed=6)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("n", [1, 3, 40, 100])
@pytest.mark.parametrize("room", [True, False])
def test_one_key_gives_its_value(cuda_lib, form, n, room):
    """A row that sees one key has that key's value, for every code and for scales
    from the least to the largest that the store writes: nothing is rounded on the
    way to O.  Row i sees key i alone (a window of one)."""
    code, dtype = form
    for e in (quant64.LEAST[form], -9, 0, 7) + ((60, 119) if dtype == BF16 else ()):
        c = Case([(n, n)], Hq=2, Hkv=1, form=form, block=1, kind=SLIDING, window=1, sink=False)
        num = torch.arange(256, dtype=torch.uint8)
        num[127 if code == "e4m3" else 128] = 0
        if code == "e4m3":
            num[255] = 0
        rows = torch.stack([num[:128], num[128:]])[torch.arange(16) % 2]   # of a page
        pages = rows.view(1, 1, 16, 128).expand(c.cache.k_pages.shape)
        c.cache.v_pages.view(torch.uint8).copy_(pages)
        c.cache.v_scales.fill_(e + 127)
        (o, lse), status = c.run(room)
        assert status == mab.ATTN_OK
        want = rows.view(quant64.TYPES[code]).float()[torch.arange(n) % 16].double() * 2.0 ** e
        assert torch.equal(o.cpu().double(), want[:, None].expand(n, 2, 128))


@pytest.mark.parametrize("n", [1, 40, 100])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_query_magnitudes(cuda_lib, size, n):
    """bf16 queries of any size over keys of the opposite one."""
    c = Case([(n, 200)], form=("e4m3", BF16), block=16, spread=0)
    e = round(math.log2(size))
    c.q.mul_(size)
    for s, k in ((c.cache.k_scales, c.k),):
        s.copy_(torch.where(s == 255, s, s - e) if abs(e) < 100 else
                torch.where(s == 255, s, (s.int() - e).clamp(1, 254).to(torch.uint8)))
        k[0].mul_(2.0 ** -e)
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_query_rows_not_finite(cuda_lib, n):
    """A row of q that is not finite gives NaN in its own o and lse alone."""
    c = Case([(n, 400), (1, 90)], Hq=4, Hkv=1, form=("e4m3", BF16))
    (o0, l0), _ = c.run()
    c.q[0, 2, 5] = float("nan")
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    assert bool(torch.isnan(o[0, 2]).all()) and bool(torch.isnan(lse[2, 0]))
    o[0, 2], lse[2, 0] = o0[0, 2], l0[2, 0]
    assert torch.equal(o, o0) and torch.equal(lse, l0)


@pytest.mark.parametrize("n", [1, 20, 200])
@pytest.mark.parametrize("room", [True, False])
def test_captured_with_other_lengths(cuda_lib, n, room):
    a = Case([(n, 1000), (n, 264), (n, 2000)], ps=32, form=("e4m3", F16), seed=1)
    ws = a.workspace(room)
    out = (torch.full_like(a.q, 7.0), torch.full((a.Hq, a.T), 7.0, device="cuda"))
    call = lambda: mab.paged_fwd(a.q, a.cache, a.table, a.sink, a.mask, SCALE, ws=ws, out=out)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    b = Case([(n, 300), (n, 1999), (n, 251)], ps=32, form=("e4m3", F16), seed=2)
    P = b.cache.num_pages
    assert P <= a.cache.num_pages
    for x, y in ((a.cache.k_pages, b.cache.k_pages), (a.cache.v_pages, b.cache.v_pages)):
        x.view(torch.uint8)[:P].copy_(y.view(torch.uint8)[:P])
    for x, y in ((a.cache.k_scales, b.cache.k_scales), (a.cache.v_scales, b.cache.v_scales)):
        x[:P].copy_(y[:P])
    cols = min(a.table.shape[1], b.table.shape[1])
    a.table[:, :cols].copy_(b.table[:, :cols])
    a.lens.copy_(b.lens)
    a.q.copy_(b.q)
    a.sink.copy_(b.sink)
    g.replay()
    torch.cuda.synchronize()
    assert mab.device_status(ws) == mab.ATTN_OK
    b.check(*out)


def test_repeats_are_equal(cuda_lib):
    for n, room in ((1, True), (3, True), (12, True), (70, True), (70, False)):
        c = Case([(n, 5000), (n, 900), (n, 77)], Hq=8, Hkv=2, ps=32, seed=n)
        (o0, l0), _ = c.run(room)
        for _ in range(5):
            (o, lse), _ = c.run(room)
            assert torch.equal(o, o0) and torch.equal(lse, l0)


@pytest.mark.parametrize("reqs,Hq,Hkv,window,code", [
    ([(500, 9826)] + [(1 + i % 4, 1700 + 900 * i) for i in range(15)], 32, 8, 1024, "e4m3"),
    ([(5, 60000), (4, 50000)], 32, 4, 0, "i8"),
    ([(1, 3000 + 1000 * i) for i in range(12)], 32, 8, 0, "e4m3")])
def test_repeats_are_equal_from_cold_memory(cuda_lib, monkeypatch, reqs, Hq, Hkv, window, code):
    """Calls one behind another over caches that push one another out of the L2, so
    that loads arrive late and out of their order."""
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM")
    g = torch.Generator("cuda").manual_seed(3)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ps = 32
    held = [-(-L // ps) for _, L in reqs]
    new = [n for n, _ in reqs]
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    mask = mab.Mask(kind=FIRST if window else CAUSAL, window=window, first=4 if window else 0,
                    cu_seqlens_q=i(cu), seqlen_k=i([L for _, L in reqs]), total_q=sum(new),
                    max_seqlen_q=max(new), max_seqlen_k=max(L for _, L in reqs))
    states = []
    for _ in range(3):
        P = sum(held) + 900
        cache = mab.PagedCache8.empty(P, Hkv, ps, 1, torch.int8 if code == "i8" else
                                      torch.float8_e4m3fn, F16, "NHD")
        for t in (cache.k_pages, cache.v_pages):
            u = torch.randint(0, 120, t.shape, generator=g, device="cuda", dtype=torch.uint8)
            t.view(torch.uint8).copy_(u | torch.randint(0, 2, t.shape, generator=g, device="cuda",
                                                        dtype=torch.uint8) << 7)
        for t in (cache.k_scales, cache.v_scales):
            t.copy_(torch.randint(116, 121, t.shape, generator=g, device="cuda"))
        ids = torch.randperm(P, generator=g, device="cuda").int()
        table = torch.zeros(len(reqs), max(held), dtype=torch.int32, device="cuda")
        for b, h in enumerate(held):
            table[b, :h] = ids[sum(held[:b]):sum(held[:b]) + h]
        q = torch.randn(sum(new), Hq, 128, generator=g, device="cuda").to(F16)
        states.append((q, cache, table))
    run = lambda st: mab.paged_fwd(st[0], st[1], st[2], None, mask, SCALE)
    first = [run(st) for st in states]
    for _ in range(8):
        again = [run(states[k % 3]) for k in range(48)]
        for k, (o, lse) in enumerate(again):
            assert torch.equal(o, first[k % 3][0]) and torch.equal(lse, first[k % 3][1])
        del again


def test_no_lse_and_other_stream(cuda_lib):
    c = Case([(1, 300), (70, 100)], form=("i8", BF16))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, lse = mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, stream=st)
    st.synchronize()
    c.check(o, lse)
    out = torch.empty_like(c.q)
    mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, out=(out, None))
    assert torch.equal(out, o)


@pytest.mark.parametrize("n", [1, 40, 200])
def test_waits_that_run_out(cuda_lib, n, monkeypatch):
    """The loader issues nothing: the call ends with a status."""
    c = Case([(n, 500)])
    monkeypatch.setenv("MASKATTN_TEST_NO_LOADS", "1")
    monkeypatch.setenv("MASKATTN_WAIT_TIMEOUT_NS", "20000000")
    _, status = c.run()
    monkeypatch.delenv("MASKATTN_TEST_NO_LOADS")
    monkeypatch.delenv("MASKATTN_WAIT_TIMEOUT_NS")
    assert status == mab.ATTN_ERR_TIMEOUT
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)
