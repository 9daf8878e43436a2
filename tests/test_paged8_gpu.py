"""Stores into the 8-bit cache and rows read back, against the plain form in 64
bits: codes, scales and values are equal, not close."""
import random

import pytest
import torch

import quant64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
FORMS = [("e4m3", F16), ("e4m3", BF16), ("i8", F16), ("i8", BF16)]
IDS = ["e4m3-f16", "e4m3-bf16", "i8-f16", "i8-bf16"]


class Store:
    """A cache of P pages in both forms, and steps of new tokens at slots."""

    def __init__(self, kind, dtype, P=6, Hkv=3, ps=32, block=16, layout="HND", seed=0):
        self.plain = [quant64.Cache64(P, Hkv, ps, block, kind, dtype) for _ in range(2)]
        self.g = torch.Generator("cpu").manual_seed(seed)
        self.kind, self.dtype, self.Hkv, self.layout, self.ps, self.P = kind, dtype, Hkv, layout, \
            ps, P
        # what earlier owners of the pages left: any codes, any scales
        self.cache = mab.PagedCache8.empty(P, Hkv, ps, block, quant64.TYPES[kind], dtype, layout)
        for c in (self.cache.k_pages, self.cache.v_pages):
            junk = torch.randint(0, 127, c.shape, generator=self.g, dtype=torch.uint8)
            c.view(torch.uint8).copy_(junk)
        for s, p in ((self.cache.k_scales, self.plain[0]), (self.cache.v_scales, self.plain[1])):
            junk = torch.randint(100, 150, s.shape, generator=self.g, dtype=torch.uint8)
            s.copy_(junk)
            p.exp.copy_(junk.long() - 127)
        for c, p in ((self.cache.k_pages, self.plain[0]), (self.cache.v_pages, self.plain[1])):
            n = c.cpu().float().double()
            p.num.copy_(n if layout == "NHD" else n.transpose(1, 2))

    def rows(self, T, size=1.0):
        x = torch.randn(T, self.Hkv, 128, generator=self.g) * size
        return x.to(self.dtype)

    def step(self, k, v, slots, **kw):
        s = torch.tensor(slots, dtype=torch.int64).cuda()
        mab.paged_store(self.cache, k.cuda(), v.cuda(), s, **kw)
        for p, x in zip(self.plain, (k, v)):
            p.store(x, slots)

    def check(self):
        torch.cuda.synchronize()
        for name, c, s, p in (("k", self.cache.k_pages, self.cache.k_scales, self.plain[0]),
                              ("v", self.cache.v_pages, self.cache.v_scales, self.plain[1])):
            assert torch.equal(s.cpu(), p.bytes()), f"scales of {name}"
            got = c.cpu().float().double()
            got = got if self.layout == "NHD" else got.transpose(1, 2)
            fine = (p.exp != p.BAD).repeat_interleave(p.block, 2).transpose(1, 2)[..., None]
            assert torch.equal(torch.where(fine, got, 0.0), torch.where(fine, p.num, 0.0)), name

    def read(self, slots):
        """Values of the slots through paged_load, a request of one row each."""
        n = len(slots)
        rel = [s % self.ps for s in slots]
        table = torch.tensor([[s // self.ps] for s in slots], dtype=torch.int32).cuda()
        cu = torch.arange(n + 1, dtype=torch.int32).cuda()
        return mab.paged_load(self.cache, table, cu, n,
                              torch.tensor(rel, dtype=torch.int32).cuda())


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("block,ps", [(1, 16), (1, 48), (16, 16), (16, 48), (32, 64), (64, 64),
                                      (64, 128)])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_appends(cuda_lib, kind, dtype, block, ps, layout):
    """Requests that grow by chunks and single tokens, magnitudes that change."""
    st = Store(kind, dtype, P=7, ps=ps, block=block, layout=layout, seed=ps + block)
    r = random.Random(block * ps)
    order = list(range(7))
    r.shuffle(order)
    owned = [order[:3], order[3:6]]
    at = [0, 0]
    while min(at) < 2 * ps:
        slots = []
        for b in range(2):
            n = min(r.choice([1, 1, 3, block, 2 * block + 1, ps - 1]), 3 * ps - at[b])
            slots += [owned[b][x // ps] * ps + x % ps for x in range(at[b], at[b] + n)]
            at[b] += n
        pad = r.choice([0, 2])
        slots += [-1] * pad
        size = 2.0 ** r.uniform(-6, 6)
        st.step(st.rows(len(slots), size), st.rows(len(slots), 1.0), slots)
        st.check()
    live = [owned[b][x // ps] * ps + x % ps for b in range(2) for x in range(at[b])]
    for got, p in zip(st.read(live), st.plain):
        assert torch.equal(got.cpu().double(), p.values(live))


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("block", [1, 16])
def test_magnitudes(cuda_lib, kind, dtype, block):
    """The largest and the least numbers of the types, zeros, and borders of the
    scales: all values come back finite."""
    st = Store(kind, dtype, P=8, ps=16, block=block, Hkv=2)
    f = torch.finfo(dtype)
    edge = quant64.TOP[kind]
    tops = [f.max, f.max / 2, f.tiny, f.tiny * f.eps, 0.0, edge, edge / 256, 1.0]
    k = st.rows(128, 0.25)
    for p, t in enumerate(tops):
        x = k[16 * p:16 * p + 16]
        x *= t if t > 0 else 0.0
        x.clamp_(-t, t)
        x[3, 0, 5], x[7, 1, 100] = t, -t
        x[2, :, 7] = -0.0
    v = k.flip(0).contiguous()
    st.step(k, v, list(range(128)))
    st.check()
    for got, p in zip(st.read(list(range(128))), st.plain):
        assert bool(torch.isfinite(got).all())
        assert torch.equal(got.cpu().double(), p.values(list(range(128))))


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("block", [1, 16, 32])
def test_not_finite(cuda_lib, kind, dtype, block):
    st = Store(kind, dtype, P=4, ps=32, block=block, Hkv=2)
    k, v = st.rows(40), st.rows(40)
    k[3, 0, 17] = float("nan")
    v[20, 1, 0] = float("-inf")
    k[39, 1, 127] = float("inf")
    slots = list(range(32, 72))
    st.step(k, v, slots)
    st.check()
    for got, p in zip(st.read(slots), st.plain):
        want = p.values(slots)
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(got.cpu().double().nan_to_num(5.0), want.nan_to_num(5.0))
    # later rows of such a block stay NaN, a block that begins anew does not
    st.step(st.rows(3), st.rows(3), [72, 73, 74])
    st.check()
    st.step(st.rows(32), st.rows(32), list(range(32, 64)))
    st.check()
    assert bool(torch.isfinite(st.read(list(range(32, 64)))[0]).all())


def test_slots_outside_and_strided_rows(cuda_lib):
    st = Store("e4m3", BF16, P=3, ps=16, Hkv=2)
    qkv = torch.randn(9, 6, 128, generator=st.g).to(BF16)
    slots = [5, 6, -1, 48, 2 ** 40, -2 ** 40, 17, 18, 47]
    dev = qkv.cuda()
    mab.paged_store(st.cache, dev[:, 2:4], dev[:, 4:], torch.tensor(slots).cuda())
    for p, x in zip(st.plain, (qkv[:, 2:4], qkv[:, 4:])):
        p.store(x, slots)
    st.check()


@pytest.mark.parametrize("block", [1, 16])
def test_pages_in_wider_tensors(cuda_lib, block):
    """K and V pages as halves of one tensor, their scales too."""
    both = torch.zeros(5, 2, 2, 32, 128, dtype=torch.int8).cuda()
    sb = torch.full((5, 2, 2, 32 // block), 9, dtype=torch.uint8).cuda()
    cache = mab.PagedCache8(both[:, 0], both[:, 1], sb[:, 0], sb[:, 1], F16)
    st = Store("i8", F16, P=5, ps=32, Hkv=2, block=block)
    for p in st.plain:
        p.num.zero_()
        p.exp.fill_(9 - 127)
    st.cache = cache
    st.step(st.rows(70), st.rows(70), list(range(40, 110)))
    st.check()
    for got, p in zip(st.read(list(range(40, 110))), st.plain):
        assert torch.equal(got.cpu().double(), p.values(list(range(40, 110))))


@pytest.mark.parametrize("T", [1, 31, 500, 5000, 40000])
def test_many_tokens(cuda_lib, T):
    """Every share of tokens a warp looks through."""
    ps, Hkv = 64, 4
    P = -(-T // ps) + 1
    g = torch.Generator("cuda").manual_seed(T)
    k = torch.randn(T, Hkv, 128, generator=g, device="cuda").to(BF16)
    cache = mab.PagedCache8.empty(P, Hkv, ps, 16, torch.float8_e4m3fn, BF16, "NHD")
    first = 5
    slots = torch.arange(first, first + T, device="cuda")
    cache.k_scales.fill_(1)
    cache.v_scales.fill_(1)
    cache.k_pages.view(torch.uint8).zero_()
    cache.v_pages.view(torch.uint8).zero_()
    mab.paged_store(cache, k, k, slots)
    back, _ = mab.paged_load(cache, torch.arange(P, dtype=torch.int32, device="cuda")[None],
                             torch.tensor([0, T], dtype=torch.int32, device="cuda"), T,
                             torch.tensor([first], dtype=torch.int32, device="cuda"))
    # the definition, vectorised: blocks of 16 from slot 0, the first one cut
    x = torch.zeros(P * ps, Hkv, 128, dtype=torch.float64, device="cuda")
    x[first:first + T] = k.double()
    b = x.reshape(-1, 16, Hkv, 128)
    m, e = torch.frexp(b.abs().amax((1, 3)).clamp(min=2.0 ** -100))
    e = (e - 9 + (m > 0.875).int()).double()
    want = quant64.nearest("e4m3", b / torch.exp2(e)[:, None, :, None], 448.0) * \
        torch.exp2(e)[:, None, :, None]
    assert torch.equal(back.double(), want.reshape(-1, Hkv, 128)[first:first + T])


def test_load_rules(cuda_lib):
    """Requests without rows, rows before, between and behind requests, starts,
    pages and positions that are not there."""
    st = Store("i8", F16, P=5, ps=16, Hkv=2, block=16)
    st.step(st.rows(80), st.rows(80), list(range(80)))
    table = torch.tensor([[3, 1], [0, -1], [2, 4], [9, 2]], dtype=torch.int32).cuda()
    #       rows 2..21 of request 0 from position 7; none of 1 at 22..22; 2: 22..24; 3: 25..60
    cu = torch.tensor([2, 22, 22, 25, 61], dtype=torch.int32).cuda()
    start = torch.tensor([7, 3, 15, -4], dtype=torch.int32).cuda()
    out = tuple(torch.full((70, 2, 128), 7.0, dtype=F16, device="cuda") for _ in range(2))
    mab.paged_load(st.cache, table, cu, 70, start, out=out)
    for o, p in zip(out, st.plain):
        want = torch.full((70, 2, 128), 7.0, dtype=torch.float64)
        for t in range(2, 61):
            b = 0 if t < 22 else 2 if t < 25 else 3
            x = max(int(start[b]), 0) + t - int(cu[b])
            page = int(table[b, x // 16]) if x < 32 else -1
            want[t] = p.values([page * 16 + x % 16])[0] if 0 <= page < 5 else 0.0
        assert torch.equal(o.cpu().double(), want)
    many = torch.arange(4001, dtype=torch.int32).cuda()   # one row each
    tab = (torch.arange(4000, dtype=torch.int32) % 5)[:, None].cuda()
    k, _ = mab.paged_load(st.cache, tab, many, 4000)
    first = st.plain[0].values([0, 16, 32, 48, 64])
    assert torch.equal(k.cpu().double(), first.repeat(800, 1, 1))


def test_every_code(cuda_lib):
    """All codes under scales from the least to the largest."""
    for kind, dtype in FORMS:
        least = quant64.LEAST[kind, dtype]
        st = Store(kind, dtype, P=2, ps=16, Hkv=2, block=1)
        codes = torch.arange(256, dtype=torch.uint8)
        if kind == "e4m3":
            codes[127], codes[255] = 0, 0
        else:
            codes[128] = 0
        for s in (least, -15, -9, 0, 7):
            for c in (st.cache.k_pages, st.cache.v_pages):
                c.view(torch.uint8).copy_(codes.view(2, 1, 1, 128).expand(2, 2, 16, 128))
            st.cache.k_scales.fill_(s + 127)
            st.cache.v_scales.fill_(s + 127)
            k, v = st.read([0, 16])
            num = codes.view(quant64.TYPES[kind]).float().double() * 2.0 ** s
            want = num.view(2, 1, 128).expand(2, 2, 128)
            assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), want)


def test_captured_step(cuda_lib):
    """Replayed with other slots, rows and page contents."""
    st = Store("e4m3", F16, P=4, ps=16, Hkv=2)
    k, v = st.rows(20).cuda(), st.rows(20).cuda()
    slots = torch.arange(20).cuda()
    mab.paged_store(st.cache, k, v, slots)
    for p, x in zip(st.plain, (k, v)):
        p.store(x, list(range(20)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mab.paged_store(st.cache, k, v, slots)
    k.copy_(st.rows(20, 5.0))
    v.copy_(st.rows(20, 0.1))
    slots.copy_(torch.arange(20, 40))
    g.replay()
    for p, x in zip(st.plain, (k, v)):
        p.store(x, list(range(20, 40)))
    st.check()
