"""The rules of the paged cache's calls at cases worked out by hand."""

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab
from test_paged_gpu import NONE, Case

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _plan(cached, fresh, stack, count, table, max_tokens):
    tab, free = _i32(table), _i32(stack)
    p = mab.paged_plan(_i32(cached), _i32(fresh), free, _i32([count]), tab, 16, max_tokens)
    torch.cuda.synchronize()
    names = ("cu_seqlens_q", "seqlen_k", "free_count", "slot_map", "position", "refused")
    return {**{n: getattr(p, n).tolist() for n in names}, "table": tab.tolist(),
            "stack": free.tolist()}


def test_what_can_never_be_placed_takes_no_page(cuda_lib):
    # four pages of 16 a request, three free: 100 tokens never fit a row, so
    # their seven pages do not stand in the way of the second request's one
    got = _plan([0, 0], [100, 10], [5, 2, 7, 0, 0, 0, 0, 0], 3, [[-1] * 4, [-1] * 4], 120)
    assert got == dict(cu_seqlens_q=[0, 100, 110], seqlen_k=[0, 10], free_count=[2],
                       slot_map=[-1] * 100 + list(range(112, 122)) + [-1] * 10,
                       position=list(range(100)) + list(range(10)) + [-1] * 10, refused=[1],
                       table=[[-1] * 4, [7, -1, -1, -1]], stack=[5, 2, 7, 0, 0, 0, 0, 0])


def test_a_need_that_does_not_fit_stops_the_later_ones(cuda_lib):
    # 2, 3 and 1 pages of four: the second request's do not fit, the third comes
    # after it; the fourth needs none (its 17th token has room on its page)
    got = _plan([0, 16, 16, 16 + 5], [32, 40, 1, 1], [9, 8, 6, 4] + [0] * 6, 4,
                [[-1] * 4, [1, -1, -1, -1], [2, -1, -1, -1], [3, 5, -1, -1]], 80)
    assert got == dict(cu_seqlens_q=[0, 32, 72, 73, 74], seqlen_k=[32, 16, 16, 22], free_count=[2],
                       slot_map=[64 + i for i in range(16)] + [96 + i for i in range(16)] +
                       [-1] * 41 + [5 * 16 + 5] + [-1] * 6,
                       position=list(range(32)) + list(range(16, 56)) + [16, 21] + [-1] * 6,
                       refused=[2], stack=[9, 8, 6, 4] + [0] * 6,
                       table=[[4, 6, -1, -1], [1, -1, -1, -1], [2, -1, -1, -1], [3, 5, -1, -1]])


def test_tokens_past_the_last_entry(cuda_lib):
    # the first request's 20 tokens end past 10; the second, without any, too
    got = _plan([0, 5], [20, 0], [1, 2, 3, 0], 3, [[-1] * 2, [0, -1]], 10)
    assert got == dict(cu_seqlens_q=[0, 20, 20], seqlen_k=[0, 5], free_count=[3],
                       slot_map=[-1] * 10, position=list(range(10)), refused=[2],
                       table=[[-1] * 2, [0, -1]], stack=[1, 2, 3, 0])


@pytest.mark.parametrize("L", [1, 4, 70])
def test_more_new_tokens_than_keys_without_a_rule(cuda_lib, L):
    # every row sees every key, those before position zero too
    c = Case([(90, 90)], kind=NONE, seed=L)
    c.lens.fill_(L)
    c.k[0], c.v[0], c.vis[0] = c.k[0][:L], c.v[0][:L], c.vis[0][:, :L]
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    c.check(o, lse)
    c.lens.zero_()
    (o, lse), _ = c.run()
    assert bool((o == 0).all())
    # the sink through a change of base and back: two products and their constants
    assert torch.allclose(lse, c.sink[:, None].expand_as(lse), rtol=2.0 ** -22, atol=0)
