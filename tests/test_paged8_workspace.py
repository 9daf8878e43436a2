"""Workspaces of attention over the 8-bit cache: how much the binding asks for."""
import pytest
import torch

from masked_attention_backward_gb300 import binding as mab


class Call:
    """A call that wants room by its bounds (chunks of 2048 over 9000 keys), or one that does
    not (chunks of 256 over 256).  On the host: only sizes are asked for."""

    def __init__(self, Sq=2048, Skv=9000, Hkv=8):
        e = lambda *s, dt: torch.empty(s, dtype=dt)
        self.cache = mab.PagedCache8(e(4, Hkv, 64, 128, dt=torch.int8),
                                     e(4, Hkv, 64, 128, dt=torch.int8),
                                     e(4, Hkv, 4, dt=torch.uint8), e(4, Hkv, 4, dt=torch.uint8))
        self.q = e(Sq, 2 * Hkv, 128, dt=torch.bfloat16)
        i = lambda n: torch.zeros(n, dtype=torch.int32)
        self.mask = mab.Mask(kind=mab.ATTN_MASK_CAUSAL, cu_seqlens_q=i(2), seqlen_k=i(1),
                             total_q=Sq, max_seqlen_q=Sq, max_seqlen_k=Skv)

    def sizes(self):
        sh = mab.paged_shape(self.q, self.cache, self.mask)
        return (mab.attn_paged8_workspace_size(sh)[1],
                mab.attn_paged8_workspace_size(sh, self.mask.desc())[1])

    def given(self):
        return mab.paged_workspace(self.q, self.cache, self.mask).numel()


def test_the_hook_holds_from_call_to_call(monkeypatch):
    """MASKATTN_PAGED8_ROOM is read at each call, whatever an earlier call of the same
    sizes was given."""
    c = Call(256, 256)
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM", raising=False)
    least, room = c.sizes()
    assert room == least == c.given()
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    _, room = c.sizes()
    assert room > least and c.given() == room
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM")
    assert c.given() == least


def test_the_most_that_is_asked_for(monkeypatch):
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM", raising=False)
    c = Call()
    least, room = c.sizes()
    assert room > least and c.given() == room
    monkeypatch.setattr(mab, "PAGED8_ROOM", room - least - 1)
    assert c.given() == least
    monkeypatch.setattr(mab, "PAGED8_ROOM", room - least)
    assert c.given() == room


def test_the_least_where_there_is_no_memory_for_more(monkeypatch):
    monkeypatch.delenv("MASKATTN_PAGED8_ROOM", raising=False)
    c = Call()
    least, room = c.sizes()
    empty = torch.empty

    def short(n, *a, **kw):
        if n > least:
            raise torch.OutOfMemoryError("no memory")
        return empty(n, *a, **kw)

    monkeypatch.setattr(torch, "empty", short)
    assert c.given() == least
    # ... and where there is not even that, the allocator's error
    least -= 1
    with pytest.raises(torch.OutOfMemoryError):
        c.given()


@pytest.mark.gpu
def test_a_call_where_there_is_no_memory_for_more(cuda_lib, monkeypatch):
    """Goes on with the least workspace, with that workspace's results."""
    import test_paged8_fwd_gpu as fwd
    monkeypatch.setenv("MASKATTN_PAGED8_ROOM", "1")
    c = fwd.Case([(300, 700), (1, 90)], ps=32)
    (o, lse), _ = c.run(room=False)
    least = c.workspace(room=False).numel()
    assert c.workspace().numel() > least
    empty, refused = torch.empty, []

    def short(*a, **kw):
        if kw.get("dtype") == torch.uint8 and a[0] > least:
            refused.append(a[0])
            raise torch.OutOfMemoryError("no memory")
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", short)
    got = mab.paged_fwd(c.q, c.cache, c.table, c.sink, c.mask, fwd.SCALE)
    assert refused and torch.equal(got[0], o) and torch.equal(got[1], lse)
    c.check(*got)
