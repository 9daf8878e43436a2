"""Attention over a paged cache against a plain 64-bit implementation, one
request and head at a time.  Unless a test says otherwise the pages hold NaN
wherever no new token sees a key, and the table holds -7 there."""
import math
import random

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SCALE = 1.0 / math.sqrt(128)
NONE, CAUSAL, SLIDING, FIRST = (mab.ATTN_MASK_NONE, mab.ATTN_MASK_CAUSAL, mab.ATTN_MASK_SLIDING,
                                mab.ATTN_MASK_SLIDING_FIRST)


class Case:
    """reqs: (new tokens, keys) of each request."""

    def __init__(self, reqs, Hq=4, Hkv=2, ps=16, layout="HND", dtype=BF16, kind=CAUSAL, window=0,
                 first=0, sink=True, seed=0, pad=0, spare_cols=1):
        g = torch.Generator("cpu").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.reqs, self.kind, self.window, self.first = reqs, kind, window, first
        self.Hq, self.Hkv, self.ps, self.dtype = Hq, Hkv, ps, dtype
        held = [-(-L // ps) for _, L in reqs]
        P, cols = sum(held) + 3, max(held) + spare_cols
        ids = list(range(P))
        random.Random(seed).shuffle(ids)
        kp = torch.full((P, ps, Hkv, 128), float("nan"))
        vp = torch.full((P, ps, Hkv, 128), float("nan"))
        table = torch.full((len(reqs), cols), -7, dtype=torch.int32)
        self.k, self.v, self.vis = [], [], []
        at = 0
        for b, (n, L) in enumerate(reqs):
            k, v = r(L, Hkv, 128), r(L, Hkv, 128)
            x = torch.arange(L - n, L)
            j = torch.arange(L)
            vis = attn64.window_first(x, j, None if kind == CAUSAL else window,
                                      first if kind == FIRST else 0)
            if kind == NONE:
                vis = torch.ones(n, L, dtype=torch.bool)
            seen = vis.any(0)
            for c in range(held[b]):
                rows = torch.arange(c * ps, min((c + 1) * ps, L))
                if bool(seen[rows].any()):
                    table[b, c] = ids[at]
                    live = rows[seen[rows]]
                    kp[ids[at], live - c * ps] = k[live]
                    vp[ids[at], live - c * ps] = v[live]
                at += 1
            self.k.append(k.to(dtype).cuda())
            self.v.append(v.to(dtype).cuda())
            self.vis.append(vis.cuda())
        if layout == "HND":
            kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
        self.cache = mab.PagedCache(kp.to(dtype).contiguous().cuda(),
                                    vp.to(dtype).contiguous().cuda(), layout)
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

    def run(self, **kw):
        ws = mab.paged_workspace(self.q, self.cache, self.mask)
        ws.fill_(0xff)
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


def _go(*a, **kw):
    c = Case(*a, **kw)
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 640, 1001])
def test_one_token(cuda_lib, L, dtype):
    _go([(1, L)], dtype=dtype, sink=L % 2 == 0, seed=L)


@pytest.mark.parametrize("n,L", [(1, 1), (2, 2), (3, 70), (64, 64), (65, 65), (127, 300),
                                 (130, 130), (200, 1000), (500, 500)])
@pytest.mark.parametrize("kind,window,first", [(CAUSAL, 0, 0), (SLIDING, 1, 0), (SLIDING, 70, 0),
                                               (FIRST, 40, 3), (FIRST, 100, 130), (NONE, 0, 0)])
def test_chunks(cuda_lib, n, L, kind, window, first):
    _go([(n, L)], kind=kind, window=window, first=first, seed=n + L, pad=3)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (6, 2), (10, 2), (7, 1), (16, 1), (33, 1),
                                    (64, 1), (128, 1), (100, 1), (32, 8)])
def test_head_groups(cuda_lib, Hq, Hkv):
    _go([(1, 200), (30, 90), (5, 5)], Hq=Hq, Hkv=Hkv, seed=Hq)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 96, 112, 128, 208, 1024])
def test_page_sizes(cuda_lib, ps, layout):
    _go([(1, 333), (40, 555), (1, ps), (2, ps + 1)], ps=ps, layout=layout, dtype=F16, seed=ps)
    _go([(3, 700), (70, 1300)], ps=ps, layout=layout, kind=FIRST, window=100, first=20, seed=ps)


def test_ragged_batch(cuda_lib):
    r = random.Random(3)
    reqs = [(0, 0), (1, 1), (0, 50), (300, 300), (1, 2000), (7, 9), (0, 0)]
    for _ in range(60):
        n = r.choice([0, 1, 1, 1, 2, 5, r.randint(1, 90)])
        reqs.append((n, n + r.choice([0, 1, r.randint(0, 900)])))
    reqs.append((0, 10))
    _go(reqs, Hq=8, Hkv=2, ps=32, seed=5, pad=9)
    _go(reqs, Hq=8, Hkv=2, ps=32, kind=FIRST, window=64, first=5, seed=6)


def test_many_requests(cuda_lib):
    r = random.Random(4)
    _go([(r.choice([0, 1, 1, 2]), r.randint(2, 150)) for _ in range(1100)], Hq=2, Hkv=1, seed=7)


@pytest.mark.parametrize("B,Hq,Hkv,L", [(1, 8, 1, 9000), (1, 32, 2, 5000), (2, 1, 1, 20000),
                                        (1, 128, 1, 6000)])
def test_long_context_in_pieces(cuda_lib, B, Hq, Hkv, L):
    _go([(1 + b, L - 7 * b) for b in range(B)], Hq=Hq, Hkv=Hkv, ps=64, seed=L)


def test_more_new_tokens_than_keys(cuda_lib):
    # positions below zero see nothing: O = 0, LSE = the sink or +inf
    for sink in (True, False):
        c = Case([(9, 9), (70, 70)], sink=sink, seed=8)
        c.lens.copy_(torch.tensor([4, 0], dtype=torch.int32))
        (o, lse), status = c.run()
        assert status == mab.ATTN_OK
        assert bool((o[:5] == 0).all()) and bool((o[9:] == 0).all())
        want = c.sink if sink else torch.full((c.Hq,), math.inf, device="cuda")
        for rows in (lse[:, :5], lse[:, 9:]):
            assert torch.allclose(rows, want[:, None].expand_as(rows), rtol=1e-6, atol=1e-6)
        assert bool(torch.isfinite(o[5:9].float()).all()) and bool((o[5:9] != 0).any())


def test_lengths_are_clamped(cuda_lib):
    c = Case([(3, 40), (2, 20)], seed=9)
    (want, wl), _ = c.run()
    # offsets past the rows, keys past the table's columns and negative ones
    c.cu.copy_(torch.tensor([0, 3, 2 ** 31 - 1], dtype=torch.int32))
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want) and torch.equal(lse, wl)
    c.lens.copy_(torch.tensor([-5, 20], dtype=torch.int32))
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o[3:], want[3:]) and bool((o[:3] == 0).all())
    c.lens.copy_(torch.tensor([2 ** 31 - 1, 20], dtype=torch.int32))
    (o, lse), status = c.run()
    assert torch.equal(o[3:], want[3:])   # (request 0 runs into entries of -7)


def test_bad_pages_read_as_zeros(cuda_lib):
    c = Case([(2, 100), (1, 70)], sink=False, seed=10, dtype=F16)
    for bad in (-1, c.cache.num_pages, 2 ** 31 - 1, -2 ** 31 + 1):
        (want, _), status = c.run()
        assert status == mab.ATTN_OK
        keep = c.table.clone()
        c.table[0, 2] = bad
        (o, lse), status = c.run()
        assert status == mab.ATTN_ERR_INVALID_ARG
        assert torch.equal(o[2:], want[2:])
        k, v = c.k[0].clone(), c.v[0].clone()
        c.k[0][32:48], c.v[0][32:48] = 0, 0
        c.check(o, lse)
        c.k[0], c.v[0] = k, v
        c.table.copy_(keep)
        (o, _), status = c.run()   # the next call starts clean
        assert status == mab.ATTN_OK and torch.equal(o, want)


def test_spread_logits(cuda_lib):
    # row maxima that keep growing along the context: the running maximum moves many times
    c = Case([(1, 3000), (20, 800)], Hq=4, Hkv=1, seed=11, sink=True)
    for b, (n, L) in enumerate(c.reqs):
        up = torch.linspace(0, 1, L, device="cuda")[:, None, None]
        t0 = int(c.cu[b])
        c.k[b].copy_((c.k[b].float() * 0.3 + 6 * up * c.q[t0, 0].float().sign()).to(c.dtype))
        for i in range(-(-L // 16)):
            rows = c.k[b][16 * i:16 * i + 16]
            c.cache.k_pages[int(c.table[b, i]), :, :rows.shape[0]] = rows.transpose(0, 1)
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)


def test_sinks(cuda_lib):
    # a sink far above and far below every logit, and none
    c = Case([(3, 90), (1, 400)], Hq=4, Hkv=1, seed=12)
    c.sink.copy_(torch.tensor([80.0, -80.0, -math.inf, 5.0]))
    (o, lse), _ = c.run()
    c.check(o, lse)


def test_repeats_bit_for_bit_and_in_a_graph(cuda_lib):
    c = Case([(1, 7000), (33, 400), (1, 900)], Hq=8, Hkv=2, ps=32, seed=13)
    (want, wl), _ = c.run()
    (o, lse), _ = c.run()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    ws = mab.paged_workspace(c.q, c.cache, c.mask)
    out = (torch.empty_like(want), torch.empty_like(wl))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, ws=ws, out=out)
    for _ in range(2):
        out[0].fill_(9), out[1].fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], wl)
    # the same graph at other lengths: shorter contexts of the same requests
    c.lens.copy_(torch.tensor([3000, 399, 17], dtype=torch.int32))
    (want, wl), _ = c.run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want) and torch.equal(out[1], wl)


def test_streams_and_outputs(cuda_lib):
    c = Case([(1, 3000), (4, 50)], seed=14)
    (want, wl), _ = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    out = torch.empty_like(want)
    mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, out=(out, None))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_new_tokens(cuda_lib):
    c = Case([(0, 5), (0, 0)], seed=15)
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and o.numel() == 0
    c = Case([(0, 5), (0, 0)], seed=15, pad=4)   # rows of q, none of a request
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)


def test_wide_table_and_sliced_cache(cuda_lib):
    c = Case([(1, 300), (20, 333)], ps=16, seed=16)
    (want, wl), _ = c.run()
    wide = torch.full((2, c.table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    P = c.cache.num_pages
    both = torch.full((P, 2, c.Hkv, c.ps, 128), float("nan"), dtype=c.dtype, device="cuda")
    both[:, 0], both[:, 1] = c.cache.k_pages, c.cache.v_pages
    c.cache = mab.PagedCache(both[:, 0], both[:, 1])
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want) and torch.equal(lse, wl)


def test_cache_past_32_bit_offsets(cuda_lib):
    # pages 2^30 elements apart: the used ones lie past 2^32 elements
    ps, Hkv, n, L = 64, 2, 3, 150
    c = Case([(n, L)], Hq=4, Hkv=Hkv, ps=ps, dtype=F16, seed=17)
    (want, wl), _ = c.run()
    step = 2 ** 30
    base = torch.empty(6 * step, dtype=F16, device="cuda")
    page = Hkv * ps * 128
    shape, strides = (6, Hkv, ps, 128), (step, ps * 128, 128, 1)
    kp, vp = torch.as_strided(base, shape, strides), torch.as_strided(base, shape, strides, page)
    for i, to in enumerate((5, 0, 4)):
        src = int(c.table[0, i])
        kp[to], vp[to] = c.cache.k_pages[src], c.cache.v_pages[src]
        c.table[0, i] = to
    c.cache = mab.PagedCache(kp, vp)
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want) and torch.equal(lse, wl)


def test_wait_that_runs_out_is_reported(cuda_lib, monkeypatch):
    c = Case([(1, 3000), (40, 300)], seed=18)
    (want, wl), _ = c.run()
    monkeypatch.setenv("MASKATTN_TEST_NO_LOADS", "1")
    monkeypatch.setenv("MASKATTN_WAIT_TIMEOUT_NS", "20000000")
    _, status = c.run()
    assert status == mab.ATTN_ERR_TIMEOUT
    monkeypatch.delenv("MASKATTN_TEST_NO_LOADS")
    monkeypatch.delenv("MASKATTN_WAIT_TIMEOUT_NS")
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("window,first", [(0, 0), (48, 4)])
def test_serving_run(cuda_lib, window, first):
    """Prompts in chunks, then decoding, with requests that come and go: plan,
    store and attention of each step, against attention over all keys so far."""
    ps, Hq, Hkv, B, cols, P = 16, 8, 2, 5, 20, 60
    r = random.Random(window)
    g = torch.Generator("cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    nan = float("nan")
    kp = torch.full((P, Hkv, ps, 128), nan, dtype=BF16, device="cuda")
    cache = mab.PagedCache(kp, kp.clone())
    stack = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    T = 64
    plan = mab.PagedPlan.empty(B, T, "cuda")
    plan.seqlen_k.zero_()
    plan.free_count.fill_(P)
    sink = torch.randn(Hq, generator=g, device="cuda")
    keys = [torch.empty(0, Hkv, 128, dtype=BF16, device="cuda") for _ in range(B)]
    vals = [x.clone() for x in keys]
    kind = FIRST if first else CAUSAL
    for step in range(14):
        fresh = []
        for b in range(B):
            L = keys[b].shape[0]
            if L > 120 and r.random() < 0.4:
                fresh.append(-1)
            else:
                fresh.append(r.choice([0, 1, 1, r.randint(1, 25 if L == 0 else 8)]))
        n_tok = sum(max(f, 0) for f in fresh)
        assert n_tok <= T
        q, k, v = randn(T, Hq, 128), randn(T, Hkv, 128), randn(T, Hkv, 128)
        mab.paged_plan(plan.seqlen_k, torch.tensor(fresh, dtype=torch.int32, device="cuda"), stack,
                       plan.free_count, table, ps, T, out=plan)
        mab.paged_store(cache, k, v, plan.slot_map)
        mask = mab.paged_mask(kind, plan, T, 25, cols * ps, window=window, first=first)
        out = (torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda"))
        mab.paged_fwd(q, cache, table, sink, mask, SCALE, out=out)
        torch.cuda.synchronize()
        assert int(plan.refused) == 0
        t0 = 0
        for b, f in enumerate(fresh):
            if f < 0:
                keys[b], vals[b] = keys[b][:0], vals[b][:0]
                continue
            keys[b] = torch.cat([keys[b], k[t0:t0 + f]])
            vals[b] = torch.cat([vals[b], v[t0:t0 + f]])
            L = keys[b].shape[0]
            i = torch.arange(L - f, L, device="cuda")
            vis = attn64.window_first(i, torch.arange(L, device="cuda"), window or None, first)
            for h in range(Hq):
                ro, rl, ob, lb = attn64.head_fwd(q[t0:t0 + f, h], keys[b][:, h // 4],
                                                 vals[b][:, h // 4], vis, float(sink[h]), SCALE)
                attn64.check("o", out[0][t0:t0 + f, h], ro, ob)
                attn64.check("lse", out[1][h, t0:t0 + f], rl, lb)
            t0 += f
        held = sum(-(-x.shape[0] // ps) for x in keys)
        assert int(plan.free_count) == P - held
        # every page is held once or free once
        used = [int(x) for b in range(B) for x in table[b, :-(-keys[b].shape[0] // ps)]]
        assert sorted(used + stack[:P - held].tolist()) == list(range(P))


def test_two_streams_at_once(cuda_lib):
    cases = [Case([(1, 2500), (30, 200)], seed=40), Case([(2, 900)] * 9, Hq=8, seed=41),
             Case([(1, 77)] * 40, ps=32, layout="NHD", dtype=F16, seed=42)]
    want = [c.run()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [mab.paged_workspace(c.q, c.cache, c.mask) for c in cases]
    for _ in range(5):
        got = [mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, ws=w, stream=s)
               for c, w, s in zip(cases, ws, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_one_workspace_for_different_calls(cuda_lib):
    # calls of different shapes one after another on one workspace (the larger's)
    big, small = Case([(40, 3000), (1, 50)], Hq=8, Hkv=1, seed=43), Case([(1, 4000)], seed=44)
    want = [c.run()[0] for c in (big, small)]
    ws = mab.paged_workspace(big.q, big.cache, big.mask)
    for _ in range(3):
        for c, w in zip((big, small), want):
            o, lse = mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, SCALE, ws=ws)
            torch.cuda.synchronize()
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("reqs", [[(1, 40), (3, 90), (70, 300)], [(1, 6000), (1, 9)]])
def test_a_query_that_is_not_finite_gives_nan(cuda_lib, reqs, bad):
    # in its own row, whole or in pieces, and in no other
    c = Case(reqs, seed=50)
    (o, lse), _ = c.run()
    for t, h in ((0, 1), (c.T - 1, 2)):
        c.q[t, h, 5] = bad
        (o2, lse2), status = c.run()
        assert status == mab.ATTN_OK
        assert bool(o2[t, h].isnan().all()) and bool(lse2[h, t].isnan())
        o2[t, h], lse2[h, t] = o[t, h], lse[h, t]
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        c.q[t, h, 5] = 0.5
        (o, lse), _ = c.run()


@pytest.mark.parametrize("B,Hq,Hkv", [(353, 8, 2), (705, 4, 1), (4096, 1, 1)])
def test_more_requests_than_threads(cuda_lib, B, Hq, Hkv):
    # several requests a thread where the work is laid out: requests without new
    # tokens, without keys, with several query tiles, with long contexts
    r = random.Random(B)
    reqs = []
    for b in range(B):
        n = r.choice([0, 1, 1, 1, 2, 5])
        reqs.append((n, n + r.choice([0, 0, 3, 40, 64, 130])))
    for b in (0, 31, 32, B // 2, B - 1):
        reqs[b] = (300, 420)
    reqs[7], reqs[B - 2] = (1, 5000), (0, 0)
    _go(reqs, Hq=Hq, Hkv=Hkv, ps=64 if B > 1000 else 16, seed=B)
