"""Tensors that a call on another stream makes (outputs and workspace): their
memory must not be handed out, or still be in use, in the order of the current
stream."""
import math

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)
S, HQ, HKV = 512, 8, 2
MASK = mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=100, first=4)


def _data():
    g = torch.Generator("cpu").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).half().cuda()
    return r(1, HQ, S, 128), r(1, HKV, S, 128), r(1, HKV, S, 128), r(1, HQ, S, 128)


def _calls():
    """name -> call(stream) returning the tensors that it made."""
    q, k, v, dO = _data()
    o, lse = mab.fwd(q, k, v, None, MASK, SCALE)
    qp = q[0].transpose(0, 1).contiguous()
    cache = mab.PagedCache(k[0].reshape(HKV, S // 64, 64, 128).transpose(0, 1).contiguous(),
                           v[0].reshape(HKV, S // 64, 64, 128).transpose(0, 1).contiguous())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = i32([list(range(S // 64))])
    pm = mab.Mask(kind=MASK.kind, window=100, first=4, cu_seqlens_q=i32([0, S]), seqlen_k=i32([S]),
                  total_q=S, max_seqlen_q=S, max_seqlen_k=S)
    cached, fresh, stack, count = i32([0] * 300), i32([9] * 300), i32(list(range(300))), i32([300])
    ptab = torch.zeros(300, 4, dtype=torch.int32, device="cuda")

    def plan(s):
        p = mab.paged_plan(cached, fresh, stack, count, ptab, 16, 300 * 9, stream=s)
        return p.slot_map, p.position, p.seqlen_k, p.cu_seqlens_q

    return {"fwd": lambda s: mab.fwd(q, k, v, None, MASK, SCALE, stream=s),
            "bwd": lambda s: mab.bwd(q, k, v, o, dO, lse, None, MASK, SCALE, stream=s)[:3],
            "paged_fwd": lambda s: mab.paged_fwd(qp, cache, table, None, pm, SCALE, stream=s),
            "paged_plan": plan}


@pytest.mark.parametrize("name", ["fwd", "bwd", "paged_fwd", "paged_plan"])
def test_outputs_take_no_memory_in_use_on_the_current_stream(cuda_lib, name):
    call, side = _calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while a fill of them is still to run
    torch.cuda._sleep(100_000_000)
    for t in want:
        for _ in range(3):
            x = torch.empty_like(t)
            x.fill_(7)
            del x
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name,entry,arg", [("fwd", "attn_fwd", 9), ("bwd", "attn_bwd", 14),
                                            ("paged_fwd", "attn_paged_fwd", 13)])
def test_a_call_s_workspace_is_not_handed_out_while_it_runs(cuda_lib, monkeypatch, name, entry,
                                                            arg):
    call, side = _calls()[name], torch.cuda.Stream()
    call(None)
    torch.cuda.synchronize()
    seen, real = [], getattr(mab, entry)

    def record(*a):
        seen.append((a[arg], a[arg + 1]))
        return real(*a)

    monkeypatch.setattr(mab, entry, record)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = call(side)
    (ptr, size), = seen
    blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(b.data_ptr() + size <= ptr or ptr + size <= b.data_ptr() for b in blocks)
    torch.cuda.synchronize()
    del got
