"""Rotary positions, page planning, the 8-bit cache and the attentions together, as a
server's steps and a training step use them.  Every stage is checked against its plain
form in 64 bits on what the stage before it left."""
import math

import pytest
import torch

import attn64
import quant64
from masked_attention_backward_gb300 import binding as mab
from test_rope_gpu import _angles, _check as check_rope

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SCALE = 1.0 / math.sqrt(128)


class Server:
    """B requests over a cache of P pages; step(fresh) brings fresh[b] new tokens of
    each request (negative: it ends)."""

    def __init__(self, B, P, cols, ps, block, kind, dtype, Hq=8, Hkv=2, window=90, first=3,
                 max_tokens=200, layout="HND"):
        self.B, self.ps, self.Hq, self.Hkv, self.dtype = B, ps, Hq, Hkv, dtype
        self.window, self.first, self.T = window, first, max_tokens
        self.g = torch.Generator("cpu").manual_seed(P)
        self.rp = mab.Rope(64, 10000.0, interleaved=True)
        self.cache = mab.PagedCache8.empty(P, Hkv, ps, block, quant64.TYPES[kind], dtype, layout)
        for s in (self.cache.k_scales, self.cache.v_scales):
            s.fill_(255)    # pages that were never written
        i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
        self.cached, self.fresh = i(B), i(B)
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(P, generator=self.g).to(torch.int32).cuda()
        self.count = torch.tensor([P], dtype=torch.int32, device="cuda")
        self.plan = mab.PagedPlan.empty(B, max_tokens, "cuda")
        self.qkv = torch.zeros(max_tokens, Hq + 2 * Hkv, 128, dtype=dtype, device="cuda")
        self.sink = torch.randn(Hq, generator=self.g).cuda()
        self.q, self.k = (torch.zeros(max_tokens, h, 128, dtype=dtype, device="cuda")
                          for h in (Hq, Hkv))
        self.out = (torch.zeros_like(self.q), torch.zeros(Hq, max_tokens, device="cuda"))
        self.mask = mab.paged_mask(mab.ATTN_MASK_SLIDING_FIRST, self.plan, max_tokens, max_tokens,
                                   cols * ps, window, first)
        self.ws = mab.paged_workspace(self.q, self.cache, self.mask)
        self.lens = [0] * B
        self.values = [None] * B    # per request: K and V as the cache should hold them
        self.plain = [quant64.Cache64(P, Hkv, ps, block, kind, dtype) for _ in range(2)]
        for p in self.plain:
            p.exp.fill_(p.BAD)

    def device_step(self):
        """What a graph holds: everything from the lengths on."""
        Hq, Hkv = self.Hq, self.Hkv
        mab.paged_plan(self.cached, self.fresh, self.free, self.count, self.table, self.ps, self.T,
                       out=self.plan)
        mab.rope(self.rp, self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.plan.position,
                 out=(self.q, self.k))
        mab.paged_store(self.cache, self.k, self.qkv[:, Hq + Hkv:], self.plan.slot_map)
        mab.paged_fwd(self.q, self.cache, self.table, self.sink, self.mask, SCALE, ws=self.ws,
                      out=self.out)
        self.cached.copy_(self.plan.seqlen_k)
        self.count.copy_(self.plan.free_count)

    def bring(self, fresh):
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g).to(self.dtype))

    def check(self, fresh):
        torch.cuda.synchronize()
        assert mab.device_status(self.ws) == mab.ATTN_OK and int(self.plan.refused) == 0
        Hq, Hkv = self.Hq, self.Hkv
        pos = self.plan.position.cpu()
        live = pos >= 0
        ang = _angles(self.rp, pos[live])[:, None]
        check_rope("q", self.q[live], self.rp, self.qkv[live][:, :Hq], ang, False)
        check_rope("k", self.k[live], self.rp, self.qkv[live][:, Hq:Hq + Hkv], ang, False)
        slots = self.plan.slot_map.tolist()
        for p, x in zip(self.plain, (self.k, self.qkv[:, Hq + Hkv:])):
            p.store(x, slots)
        table, t0, g = self.table.cpu(), 0, Hq // Hkv
        for b, n in enumerate(fresh):
            if n < 0:
                self.lens[b] = 0
                continue
            self.lens[b] += n
            L = self.lens[b]
            if n == 0:
                continue
            rows = [int(table[b, x // self.ps]) * self.ps + x % self.ps for x in range(L)]
            k, v = (p.values(rows).cuda() for p in self.plain)
            vis = attn64.window_first(torch.arange(L - n, L), torch.arange(L), self.window,
                                      self.first).cuda()
            for h in range(Hq):
                ro, rl, ob, lb = attn64.head_fwd(self.q[t0:t0 + n, h], k[:, h // g], v[:, h // g],
                                                 vis, float(self.sink[h]), SCALE)
                attn64.check(f"o of {b}, {h}", self.out[0][t0:t0 + n, h], ro, ob)
                attn64.check(f"lse of {b}, {h}", self.out[1][h, t0:t0 + n], rl, lb)
            t0 += n


STEPS = [[70, 3, 0, 20], [1, 1, 40, 1], [1, 1, 1, 1], [5, 60, 1, -1], [1, 1, -1, 33], [1, 0, 100, 1],
         [1, 1, 1, 1], [1, 1, 2, 1]]


@pytest.mark.parametrize("kind,dtype,ps,block,layout", [
    ("e4m3", BF16, 16, 16, "HND"), ("e4m3", F16, 32, 1, "NHD"), ("i8", BF16, 64, 64, "NHD"),
    ("i8", F16, 48, 16, "HND")])
@pytest.mark.parametrize("captured", [False, True])
def test_server_steps(cuda_lib, kind, dtype, ps, block, layout, captured):
    """Prompts, single tokens and requests that end; captured: one graph serves every
    step."""
    s = Server(4, 60, 20, ps, block, kind, dtype, layout=layout)
    graph = None
    for fresh in STEPS:
        s.bring(fresh)
        if captured and graph is None:
            # (a warm-up on lengths of zero, which change nothing)
            s.fresh.zero_()
            s.device_step()
            s.bring(fresh)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.device_step()
        graph.replay() if captured else s.device_step()
        s.check(fresh)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("S,Hq,Hkv,window,first", [(200, 4, 2, 64, 3), (65, 3, 1, 1000, 0)])
def test_training_step(cuda_lib, S, Hq, Hkv, window, first, dtype):
    """q and k turned, attention forward and backward, the gradients turned back."""
    g = torch.Generator("cpu").manual_seed(S)
    r = lambda *n: torch.randn(*n, generator=g).to(dtype).cuda()
    B = 2
    q0, k0, v, dO = r(B, Hq, S, 128), r(B, Hkv, S, 128), r(B, Hkv, S, 128), r(B, Hq, S, 128)
    sink = torch.randn(Hq, generator=g).cuda()
    rp = mab.Rope(128, scaling=mab.RopeScaling("parts", 4.0, original_length=128))
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=window, first=first)
    q, k = mab.rope(rp, q0, k0)
    o, lse = mab.fwd(q, k, v, sink, mask, SCALE)
    dq, dk, dv, dsink = mab.bwd(q, k, v, o, dO, lse, sink, mask, SCALE)
    dq0, dk0 = mab.rope_bwd(rp, dq, dk)
    ang = _angles(rp, torch.arange(S).expand(B, S))[:, None]
    check_rope("q", q, rp, q0, ang, False)
    check_rope("k", k, rp, k0, ang, False)
    vis = lambda b: attn64.window_first(torch.arange(S), torch.arange(S), window, first).cuda()
    ro, rl, ob, lb = attn64.forward(q, k, v, vis, sink, SCALE)
    attn64.check("o", o, ro, ob)
    attn64.check("lse", lse, rl, lb)
    ref = attn64.backward(q, k, v, o, dO, lse, vis, sink, SCALE)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv), ("dsink", dsink)):
        attn64.check(n, t, *ref[n])
    check_rope("dq0", dq0, rp, dq, ang, True)
    check_rope("dk0", dk0, rp, dk, ang, True)


def test_two_streams_at_once(cuda_lib):
    """Two servers' steps on two streams, their own workspaces and caches."""
    a = Server(4, 60, 20, 16, 16, "e4m3", BF16)
    b = Server(4, 61, 20, 32, 1, "i8", F16)
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for fresh in STEPS[:4]:
        for s in (a, b):
            s.bring(fresh)
        torch.cuda.synchronize()
        for s, t in zip((a, b), st):
            with torch.cuda.stream(t):
                s.device_step()
        torch.cuda.synchronize()
        for s in (a, b):
            s.check(fresh)
