"""Attention over the paged cache: page numbers, sinks and queries of extreme
values."""
import math

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab
from test_paged_gpu import F16, NONE, SCALE, SLIDING, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reqs,entry", [([(2, 100), (1, 70)], 2), ([(1, 1), (1, 70)], 0),
                                        ([(1, 4000), (1, 70)], 249)])
def test_the_lowest_page_number_is_a_bad_page(cuda_lib, reqs, entry):
    c = Case(reqs, sink=False, seed=10, dtype=F16)
    (want, _), status = c.run()
    assert status == mab.ATTN_OK
    keep = c.table.clone()
    c.table[0, entry] = -2 ** 31
    (o, lse), status = c.run()
    assert status == mab.ATTN_ERR_INVALID_ARG
    n = reqs[0][0]
    assert torch.equal(o[n:], want[n:])
    rows = slice(16 * entry, 16 * entry + 16)
    c.k[0][rows], c.v[0][rows] = 0, 0
    c.check(o, lse)
    c.table.copy_(keep)
    (o, _), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want)


def test_unseen_entries_are_not_looked_at(cuda_lib):
    # whatever they hold, the lowest number too
    c = Case([(3, 900)], kind=SLIDING, window=40, seed=11)
    (want, wl), status = c.run()
    assert status == mab.ATTN_OK
    c.table[c.table == -7] = -2 ** 31
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK and torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("reqs", [[(1, 40), (3, 90), (70, 300)], [(1, 6000), (1, 9)]])
def test_a_sink_that_is_not_a_number_gives_nan(cuda_lib, reqs):
    # in its own head, whole units and joined ones, and in no other
    c = Case(reqs, seed=12)
    (want, wl), _ = c.run()
    c.sink[1] = math.nan
    (o, lse), status = c.run()
    assert status == mab.ATTN_OK
    assert bool(o[:, 1].isnan().all()) and bool(lse[1].isnan().all())
    o[:, 1], lse[1] = want[:, 1], wl[1]
    assert torch.equal(o, want) and torch.equal(lse, wl)
    # rows that see no key too
    c.lens.zero_()
    (o, lse), status = c.run()
    assert bool(o[:, 1].isnan().all()) and bool(lse[1].isnan().all())
    assert bool((o[:, 0] == 0).all()) and not bool(lse[0].isnan().any())
