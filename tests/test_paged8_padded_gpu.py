"""Chunks over the 8-bit cache in calls whose q has rows that no request owns, as a
captured step has them: the longest run of new tokens and the rows of q are bounds, the
lengths are the device's.  Whatever part of the bounds the lengths use, every token's row
is written and no other."""
import pytest
import torch

from masked_attention_backward_gb300 import binding as mab
from test_paged8_fwd_gpu import SCALE, Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
FIRST = mab.ATTN_MASK_SLIDING_FIRST


def padded(reqs, Sq, total=None, **kw):
    """A case whose bounds are Sq new tokens a request and total rows of q."""
    total = len(reqs) * Sq if total is None else total
    c = Case(reqs, pad=total - sum(n for n, _ in reqs), **kw)
    c.mask.max_seqlen_q = Sq
    return c


def go(c, room=True):
    (o, lse), status = c.run(room)
    assert status == mab.ATTN_OK
    c.check(o, lse)


@pytest.mark.parametrize("reqs", [
    [(1, 700)], [(3, 400)], [(8, 90)], [(9, 200)], [(150, 150)], [(0, 300)],
    [(150, 900), (1, 500)], [(1, 640), (1, 77)], [(0, 100), (8, 300)], [(1, 1), (150, 1000)],
    [(0, 0), (0, 90)], [(8, 64), (9, 65), (1, 66), (150, 150)]],
    ids=lambda r: "-".join(str(n) for n, _ in r))
@pytest.mark.parametrize("room", [True, False])
def test_rows_that_no_request_owns(cuda_lib, monkeypatch, reqs, room):
    """Two heads a group: eight tokens are few rows."""
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    go(padded(reqs, 150, form=("e4m3", BF16), seed=len(reqs)), room)


@pytest.mark.parametrize("code,dtype", [("e4m3", F16), ("i8", BF16)])
@pytest.mark.parametrize("more", [0, 1, 40])
def test_bounds_that_leave_room_for_few_tokens_or_none(cuda_lib, monkeypatch, more, code, dtype):
    """Rows of q from which on no request but could have more than eight tokens, and one
    less: what the call's kernels share out does not follow from them."""
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    go(padded([(130, 400), (5, 300), (9, 1000)], 130, 2 * 130 + 8 + more, form=(code, dtype),
              block=1, seed=more))


def test_window(cuda_lib, monkeypatch):
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    go(padded([(2, 3000), (260, 2000)], 300, kind=FIRST, window=500, first=70, block=1))


@pytest.mark.parametrize("reqs", [[(3, 700)], [(1, 1)], [(2048, 2300)]])
def test_room_by_the_bounds(cuda_lib, monkeypatch, reqs):
    """One request, captured for prompts of 2048 tokens over 9000 keys."""
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM", raising=False)
    c = padded(reqs, 2048, Hq=8, Hkv=8, ps=32)
    c.mask.max_seqlen_k = 9000
    least = mab.attn_paged8_workspace_size(mab.paged_shape(c.q, c.cache, c.mask))[1]
    assert c.workspace().numel() > least
    go(c)


@pytest.mark.parametrize("B", [1, 2])
def test_captured(cuda_lib, monkeypatch, B):
    """One captured call, replayed for prompts, their last tokens, and nothing."""
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    Sq = 140
    kw = dict(ps=32, block=16, form=("e4m3", F16))
    a = padded([(Sq, 2300)] * B, Sq, seed=1, **kw)   # as long as the longest replay
    ws = a.workspace()
    out = (torch.empty_like(a.q), torch.empty(a.Hq, a.T, device="cuda"))
    call = lambda: mab.paged_fwd(a.q, a.cache, a.table, a.sink, a.mask, SCALE, ws=ws, out=out)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i, n in enumerate([(3, Sq), (Sq, 1), (1, 1), (0, 5), (9, 0), (Sq, Sq)]):
        b = padded([(n[j], 900 + 250 * i + 7 * j) for j in range(B)], Sq, seed=i + 2, **kw)
        for x, y in ((a.cache.k_pages, b.cache.k_pages), (a.cache.v_pages, b.cache.v_pages)):
            m = min(x.shape[0], y.shape[0])
            x.view(torch.uint8)[:m].copy_(y.view(torch.uint8)[:m])
        for x, y in ((a.cache.k_scales, b.cache.k_scales), (a.cache.v_scales, b.cache.v_scales)):
            m = min(x.shape[0], y.shape[0])
            x[:m].copy_(y[:m])
        P, cols = a.cache.num_pages, min(a.table.shape[1], b.table.shape[1])
        assert int(b.table.max()) < P and bool((b.table[:, cols:] == -7).all())
        a.table.fill_(-7)
        a.table[:, :cols].copy_(b.table[:, :cols])
        a.cu.copy_(b.cu)
        a.lens.copy_(b.lens)
        a.q.copy_(b.q)
        a.sink.copy_(b.sink)
        for t in out:
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert mab.device_status(ws) == mab.ATTN_OK
        b.check(*out)


@pytest.mark.parametrize("reqs", [[(100, 30)], [(150, 149), (9, 0), (3, 1)], [(130, 64), (1, 200)]])
@pytest.mark.parametrize("room", [True, False])
def test_more_tokens_than_keys(cuda_lib, monkeypatch, reqs, room):
    """Tokens before position zero see nothing, in every kernel."""
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    go(padded(reqs, 150, form=("i8", F16), sink=len(reqs) != 1), room)
