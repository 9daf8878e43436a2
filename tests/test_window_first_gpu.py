"""The sliding window with first keys (ATTN_MASK_SLIDING_FIRST): forward and
backward against a plain 64-bit implementation, in every layout."""
import math

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SCALE = 1.0 / math.sqrt(128)


def _inputs(B, Hq, Hkv, S, dtype, sink, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    return (r(B, Hq, S, 128), r(B, Hkv, S, 128), r(B, Hkv, S, 128), r(B, Hq, S, 128),
            torch.randn(Hq, generator=g).cuda() if sink else None)


def _vis(S, window, first, lens=None):
    def at(b):
        i = torch.arange(S, device="cuda")
        v = attn64.window_first(i, i, window, first)
        if lens is not None:
            v = v & (i[:, None] < lens[b]) & (i[None, :] < lens[b])
        return v
    return at


def _step(q, k, v, dO, sink, mask, **kw):
    o, lse = mab.fwd(q, k, v, sink, mask, SCALE)
    grads = mab.bwd(q, k, v, o, dO, lse, sink, mask, SCALE, **kw)
    torch.cuda.synchronize()
    return o, lse, grads


def _check(o, lse, grads, q, k, v, dO, sink, vis, compensated=False):
    ro, rl, ob, lb = attn64.forward(q, k, v, vis, sink, SCALE)
    attn64.check("o", o, ro, ob)
    attn64.check("lse", lse, rl, lb)
    # the backward takes the o and lse that it was given
    ref = attn64.backward(q, k, v, o, dO, lse, vis, sink, SCALE, compensated)
    for n, x in zip(("dq", "dk", "dv", "dsink"), grads):
        if x is not None:
            attn64.check(n, x, *ref[n])


# S, window, first: one token; a window of one; first keys inside a sub-tile, ending at one, past a
# key tile, longer than the window; odd sizes; first and window meeting; nearly the whole sequence
SHAPES = [(1, 1, 1), (2, 1, 1), (65, 3, 2), (200, 1, 1), (257, 64, 4), (300, 17, 64),
          (513, 100, 128), (640, 63, 65), (777, 130, 129), (1000, 128, 5), (1025, 200, 500),
          (900, 899, 3), (900, 40, 899), (384, 128, 256)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("S,window,first", SHAPES)
def test_sizes(cuda_lib, S, window, first, dtype):
    sink = (S + first) % 2 == 0
    q, k, v, dO, sk = _inputs(1, 4, 2, S, dtype, sink, S)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=window, first=first)
    _check(*_step(q, k, v, dO, sk, mask), q, k, v, dO, sk, _vis(S, window, first))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (6, 2), (3, 3)])
def test_heads_and_batches(cuda_lib, Hq, Hkv):
    q, k, v, dO, sk = _inputs(3, Hq, Hkv, 333, BF16, True, 7)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=50, first=9)
    _check(*_step(q, k, v, dO, sk, mask), q, k, v, dO, sk, _vis(333, 50, 9))


def test_compensated(cuda_lib):
    q, k, v, dO, sk = _inputs(1, 4, 1, 700, F16, True, 8)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=90, first=30)
    _check(*_step(q, k, v, dO, sk, mask, compensated=True), q, k, v, dO, sk, _vis(700, 90, 30),
           compensated=True)


@pytest.mark.parametrize("lens", [[0, 1, 300, 64], [299, 7, 130, 0]])
def test_padded_lengths(cuda_lib, lens):
    S = 300
    q, k, v, dO, sk = _inputs(len(lens), 4, 2, S, F16, True, 9)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=40, first=70, seqlen_q=ln,
                    seqlen_k=ln)
    o, lse, grads = _step(q, k, v, dO, sk, mask)
    vis = _vis(S, 40, 70, lens)
    live = torch.arange(S, device="cuda")[None, :] < ln[:, None]
    lv = live[:, None, :].expand(lse.shape)
    assert torch.all(o[~lv] == 0) and torch.all(lse[~lv] == math.inf)
    ro, rl, ob, lb = attn64.forward(q, k, v, vis, sk, SCALE)
    attn64.check("o", torch.where(lv[..., None], o.double(), 0.0),
                 torch.where(lv[..., None], ro, 0.0), ob)
    attn64.check("lse", torch.where(lv, lse.double(), 0.0), torch.where(lv, rl, 0.0), lb)
    ref = attn64.backward(q, k, v, o, dO, torch.where(lv, lse, 0.0), vis, sk, SCALE)
    for n, x in zip(("dq", "dk", "dv", "dsink"), grads):
        attn64.check(n, x, *ref[n])


def test_packed(cuda_lib):
    lens = [0, 1, 130, 257, 64, 400]
    T, Hq, Hkv = sum(lens), 4, 2
    g = torch.Generator("cpu").manual_seed(10)
    r = lambda h: torch.randn(T, h, 128, generator=g).to(BF16).cuda()
    q, k, v, dO, sk = r(Hq), r(Hkv), r(Hkv), r(Hq), torch.randn(Hq, generator=g).cuda()
    mask = mab.packed_mask(mab.ATTN_MASK_SLIDING_FIRST, lens, lens, "cuda", window=33, first=66)
    o, lse, grads = _step(q, k, v, dO, sk, mask)
    dsink, t0 = [0.0, 0.0], 0
    for n in lens:
        if n:
            cut = lambda x: x[t0:t0 + n].transpose(0, 1)[None].contiguous()
            qs, ks, vs, os, ds = cut(q), cut(k), cut(v), cut(o), cut(dO)
            ls = lse[:, t0:t0 + n][None].contiguous()
            vis = _vis(n, 33, 66)
            ro, rl, ob, lb = attn64.forward(qs, ks, vs, vis, sk, SCALE)
            attn64.check("o", os, ro, ob)
            attn64.check("lse", ls, rl, lb)
            ref = attn64.backward(qs, ks, vs, os, ds, ls, vis, sk, SCALE)
            for name, x in zip(("dq", "dk", "dv"), grads):
                attn64.check(name, cut(x), *ref[name])
            dsink[0], dsink[1] = dsink[0] + ref["dsink"][0], dsink[1] + ref["dsink"][1]
        t0 += n
    attn64.check("dsink", grads[3], *dsink)


def test_same_as_the_kinds_it_contains(cuda_lib):
    # without first keys: the window, bit for bit; a window or first keys as long as the
    # sequence: causal, bit for bit
    S = 500
    q, k, v, dO, sk = _inputs(1, 4, 2, S, F16, True, 11)
    first = mab.ATTN_MASK_SLIDING_FIRST
    pairs = [(mab.Mask(kind=first, window=70, first=0),
              mab.Mask(kind=mab.ATTN_MASK_SLIDING, window=70)),
             (mab.Mask(kind=first, window=S, first=3), mab.Mask(kind=mab.ATTN_MASK_CAUSAL)),
             (mab.Mask(kind=first, window=2 ** 31 - 1, first=3),
              mab.Mask(kind=mab.ATTN_MASK_CAUSAL)),
             (mab.Mask(kind=first, window=5, first=2 ** 31 - 1),
              mab.Mask(kind=mab.ATTN_MASK_CAUSAL))]
    for a, b in pairs:
        oa, la, ga = _step(q, k, v, dO, sk, a)
        ob, lb, gb = _step(q, k, v, dO, sk, b)
        assert torch.equal(oa, ob) and torch.equal(la, lb)
        assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_every_output_is_written_and_repeats_bit_for_bit(cuda_lib):
    S = 700
    q, k, v, dO, sk = _inputs(2, 8, 2, S, BF16, True, 12)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=64, first=20)
    o, lse = mab.fwd(q, k, v, sk, mask, SCALE)
    ws = mab.workspace(mab.shape_of(q, k), mask, "cuda")
    runs = []
    for fill in (float("nan"), 3.0):
        ws.fill_(0xff if fill != 3.0 else 0)   # whatever the workspace held
        out = (torch.full_like(q, fill), torch.full_like(k, fill), torch.full_like(v, fill),
               torch.full_like(sk, fill))
        mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws, out=out)
        torch.cuda.synchronize()
        assert mab.device_status(ws) == mab.ATTN_OK
        runs.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_backward_against_differences(cuda_lib):
    # directional derivative of sum(O * dO) with respect to q, k, v and the sink, from the 64-bit
    # forward in central differences
    S, w, f = 150, 20, 5
    q, k, v, dO, sk = _inputs(1, 2, 1, S, F16, True, 13)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=w, first=f)
    _, _, grads = _step(q, k, v, dO, sk, mask)
    vis = _vis(S, w, f)(0)

    def loss(q, k, v, sk):
        s = torch.einsum("hid,jd->hij", q[0], k[0, 0]) * SCALE
        s = s.masked_fill(~vis, -math.inf)
        s = torch.cat([s, sk[:, None, None].expand(-1, S, 1)], 2)
        p = torch.softmax(s, 2)[..., :S]
        return (torch.einsum("hij,jd->hid", p, v[0, 0]) * dO[0].double()).sum()

    base = [x.double() for x in (q, k, v, sk)]
    g = torch.Generator("cuda").manual_seed(1)
    for at, grad in enumerate(grads):
        d = torch.randn(base[at].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, dn = list(base), list(base)
        up[at], dn[at] = base[at] + h * d, base[at] - h * d
        want = float((loss(*up) - loss(*dn)) / (2 * h))
        got = float((grad.double() * d).sum())
        # the gradient's error e has a 2-norm of at most 2^-9 of the gradient's (P, dS and the
        # output are each rounded to within 2^-11), and e . d with a normal d is normal with the
        # deviation |e|: six of those, and the differences' own truncation
        assert abs(got - want) <= 6 * 2.0 ** -9 * float(grad.double().norm()) + 1e-5 * abs(want)


@pytest.mark.parametrize("Hq,Hkv,window,first", [(8, 1, 100, 130), (16, 2, 64, 1)])
def test_first_key_tiles_in_many_pieces(cuda_lib, Hq, Hkv, window, first):
    # walks of 256 steps in up to 16 pieces; in the second call a batch element that needs fewer
    # pieces than the grid has, and one that needs none
    S = 2048
    q, k, v, dO, sk = _inputs(1, Hq, Hkv, S, BF16, True, 14)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=window, first=first)
    _check(*_step(q, k, v, dO, sk, mask), q, k, v, dO, sk, _vis(S, window, first))
    lens = [700, 0, 129]
    q, k, v, dO, sk = _inputs(3, Hq, Hkv, S, F16, True, 15)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=window, first=first, seqlen_q=ln,
                    seqlen_k=ln)
    o, lse, grads = _step(q, k, v, dO, sk, mask)
    lv = (torch.arange(S, device="cuda")[None, :] < ln[:, None])[:, None, :].expand(lse.shape)
    ref = attn64.backward(q, k, v, o, dO, torch.where(lv, lse, 0.0), _vis(S, window, first, lens),
                          sk, SCALE)
    for n, x in zip(("dq", "dk", "dv", "dsink"), grads):
        attn64.check(n, x, *ref[n])


def test_captured_backward_replays(cuda_lib):
    S = 1500
    q, k, v, dO, sk = _inputs(1, 8, 2, S, BF16, True, 16)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=128, first=10)
    o, lse = mab.fwd(q, k, v, sk, mask, SCALE)
    ws = mab.workspace(mab.shape_of(q, k), mask, "cuda")
    want = mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws)
    out = tuple(torch.empty_like(x) for x in want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws, out=out)
    for _ in range(3):
        for x in out:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_wait_that_runs_out_is_reported(cuda_lib, monkeypatch):
    S = 1100
    q, k, v, dO, sk = _inputs(1, 8, 1, S, BF16, True, 17)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=128, first=10)
    o, lse = mab.fwd(q, k, v, sk, mask, SCALE)
    ws = mab.workspace(mab.shape_of(q, k), mask, "cuda")
    want = mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws)
    monkeypatch.setenv("MASKATTN_TEST_NO_LOADS", "1")
    monkeypatch.setenv("MASKATTN_WAIT_TIMEOUT_NS", "20000000")
    mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws)
    assert mab.device_status(ws) == mab.ATTN_ERR_TIMEOUT
    monkeypatch.delenv("MASKATTN_TEST_NO_LOADS")
    monkeypatch.delenv("MASKATTN_WAIT_TIMEOUT_NS")
    got = mab.bwd(q, k, v, o, dO, lse, sk, mask, SCALE, ws=ws)
    assert mab.device_status(ws) == mab.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_without_a_workspace(cuda_lib):
    S = 1100
    q, k, v, dO, sk = _inputs(1, 8, 2, S, F16, True, 19)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=100, first=7)
    o, lse, want = _step(q, k, v, dO, sk, mask)
    got = [torch.full_like(x, float("nan")) for x in want]
    stream = torch.cuda.current_stream().cuda_stream
    r = mab.attn_bwd_noalloc(mab.shape_of(q, k), *(x.data_ptr() for x in (q, k, v, o, dO, lse, sk)),
                             mask.desc(), SCALE, *(x.data_ptr() for x in got), stream)
    assert r == mab.ATTN_OK
    torch.cuda.synchronize()
    assert mab.attn_noalloc_get_device_status(stream) == mab.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_pipeline_with_uneven_runs(cuda_lib):
    # the long run's first-key tiles are not split, the short one's are: its workspace is larger
    S, H = 2048, 160
    q, k, v, dO, sk = _inputs(1, H, H, S, BF16, True, 20)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=64, first=3)
    o, lse, want = _step(q, k, v, dO, sk, mask)
    host = mab.HostBackward(1, H, H, S, S, BF16, mask, SCALE, True, "cuda", chunks=[100, 60])
    pin = lambda x: x.cpu().pin_memory()
    out = tuple(torch.empty_like(x, device="cpu").pin_memory() for x in want)
    host(dict(q=pin(q), k=pin(k), v=pin(v), o=pin(o), dO=pin(dO), lse=pin(lse), sink=pin(sk)), out)
    torch.cuda.synchronize()
    # a run's pieces differ from the whole call's: fp32 sums in another order
    for n, a, b in zip(("dq", "dk", "dv", "dsink"), out, want):
        if n in ("dq", "dsink"):
            assert torch.equal(a, b.cpu()), n
    ref = attn64.backward(q[:, :2], k[:, :2], v[:, :2], o[:, :2], dO[:, :2], lse[:, :2],
                          _vis(S, 64, 3), sk[:2], SCALE)
    last = attn64.backward(q[:, -2:], k[:, -2:], v[:, -2:], o[:, -2:], dO[:, -2:], lse[:, -2:],
                           _vis(S, 64, 3), sk[-2:], SCALE)
    for n, a in zip(("dq", "dk", "dv"), out):
        attn64.check(n, a[:, :2].cuda(), *ref[n])
        attn64.check(n, a[:, -2:].cuda(), *last[n])


@pytest.mark.parametrize("first", [4, 200])
def test_both_forms_of_the_dkdv_kernel(cuda_lib, monkeypatch, first):
    # the tiles behind the first keys, per tile and persistent: the same bits
    S = 900
    q, k, v, dO, sk = _inputs(2, 8, 4, S, BF16, True, 21)
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=70, first=first)
    runs = []
    for form in ("tile", "units"):
        monkeypatch.setenv("MASKATTN_DKDV_SCHEDULE", form)
        runs.append(_step(q, k, v, dO, sk, mask))
    monkeypatch.delenv("MASKATTN_DKDV_SCHEDULE")
    assert all(torch.equal(a, b) for a, b in zip(runs[0][2], runs[1][2]))
    _check(*runs[1], q, k, v, dO, sk, _vis(S, 70, first))


def test_two_streams_at_once(cuda_lib):
    S = 1200
    mask = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=100, first=9)
    data = [_inputs(1, 8, 2, S, F16, True, 30 + i) for i in range(3)]
    fwd = [mab.fwd(q, k, v, sk, mask, SCALE) for q, k, v, _, sk in data]
    bwd = lambda i, **kw: mab.bwd(*data[i][:3], *fwd[i][:1], data[i][3], fwd[i][1], data[i][4], mask,
                                  SCALE, **kw)
    want = [bwd(i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [mab.workspace(mab.shape_of(d[0], d[1]), mask, "cuda") for d in data]
    for _ in range(5):
        got = [bwd(i, ws=ws[i], stream=streams[i]) for i in range(3)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("kind", [mab.ATTN_MASK_CAUSAL, mab.ATTN_MASK_SLIDING,
                                  mab.ATTN_MASK_SLIDING_FIRST])
@pytest.mark.parametrize("sink", [True, False])
def test_a_query_that_is_not_finite_gives_nan(cuda_lib, kind, sink):
    # in its own row and in no other
    S = 300
    q, k, v, _, sk = _inputs(1, 4, 2, S, F16, sink, 60)
    mask = mab.Mask(kind=kind, window=90, first=5)
    o, lse = mab.fwd(q, k, v, sk, mask, SCALE)
    for i in (0, 63, 64, 211, 299):
        bad = q.clone()
        bad[0, 2, i, 7] = float("nan")
        o2, lse2 = mab.fwd(bad, k, v, sk, mask, SCALE)
        torch.cuda.synchronize()
        assert bool(o2[0, 2, i].isnan().all()) and bool(lse2.view(4, S)[2, i].isnan())
        o2[0, 2, i] = o[0, 2, i]
        lse2.view(4, S)[2, i] = lse.view(4, S)[2, i]
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
