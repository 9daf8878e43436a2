"""Rows appended to blocks of the 8-bit cache near the largest numbers of the 16-bit
type: the codes that were there, rounded again in units of the larger scale, stay
finite in it, as the new ones do.

The definition, for one block and head: a scale 2^e of the least e with amax <= TOP 2^e
(448 for e4m3, 127 for int8) or the block's own if that is larger; codes the nearest
numbers, ties to even, of magnitude at most TOP and at most that of the largest code whose
product with 2^e is finite in the type."""
import math

import pytest
import torch

import quant64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
FORMS = [("e4m3", F16), ("e4m3", BF16), ("i8", F16), ("i8", BF16)]
IDS = ["e4m3-f16", "e4m3-bf16", "i8-f16", "i8-bf16"]


def block_values(kind, dtype, runs):
    """runs: [n, 128] rows of one head, appended one run after another to one block;
    the values that the block then stands for, in 64 bits."""
    big, num, e = torch.finfo(dtype).max, None, None
    for x in runs:
        x = x.double()
        need = int(quant64.exponent(kind, dtype, x.abs().max()[None])[0])
        new = need if e is None else max(need, e)
        limit = min(quant64.TOP[kind], big / 2.0 ** new)
        rows = quant64.nearest(kind, x / 2.0 ** new, limit)
        if num is not None:
            rows = torch.cat([quant64.nearest(kind, num * 2.0 ** (e - new), limit), rows])
        num, e = rows, new
    return num * 2.0 ** e


def stored(kind, dtype, block, runs):
    """runs of rows [n, 2, 128] into one block, a call each; (k, v) read back."""
    cache = mab.PagedCache8.empty(2, 2, 64, block, quant64.TYPES[kind], dtype)
    at = 64   # the second page's first block
    for x in runs:
        s = torch.arange(at, at + x.shape[0]).cuda()
        mab.paged_store(cache, x.cuda(), (-x).cuda(), s)
        at += x.shape[0]
    n = at - 64
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    return cache, mab.paged_load(cache, torch.tensor([[1]], dtype=torch.int32).cuda(), cu, n)


def check(kind, dtype, block, runs):
    cache, (k, v) = stored(kind, dtype, block, runs)
    assert bool(torch.isfinite(k).all()) and bool(torch.isfinite(v).all())
    for h in range(2):
        want = block_values(kind, dtype, [x[:, h] for x in runs])
        assert torch.equal(k[:, h].cpu().double(), want)
        assert torch.equal(v[:, h].cpu().double(), -want)
    return cache


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("block", [16, 32, 64])
def test_appended_to_the_largest_code(cuda_lib, kind, dtype, block):
    """A block whose largest code is the type's, one exponent below the last; then the
    type's largest number: 127 becomes 63.5, whose nearest even code, 64, has no finite
    value."""
    big = torch.finfo(dtype).max
    top = math.frexp(big)[1]   # big < 2^top
    first = quant64.TOP[kind] * 2.0 ** (top - (9 if kind == "e4m3" else 7))
    x = torch.zeros(1, 2, 128, dtype=dtype)
    x[0, 0, 5], x[0, 1, 100], x[0, 0, 6], x[0, 1, 7] = first, -first, first / 2, -first / 64
    assert float(x[0, 0, 5]) == first <= big
    y = torch.zeros(1, 2, 128, dtype=dtype)
    y[0, 0, 0], y[0, 1, 1] = big, -big
    check(kind, dtype, block, [x, y])


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
@pytest.mark.parametrize("block", [16, 64])
def test_every_code_moves_up(cuda_lib, kind, dtype, block):
    """Every code of a block, moved up by one to three exponents to the last."""
    big = torch.finfo(dtype).max
    top = math.frexp(big)[1]
    codes = torch.arange(128).double() if kind == "i8" else \
        torch.cat([quant64.e4m3_numbers(), torch.zeros(1, dtype=torch.float64)])
    for up in (1, 2, 3):
        e = top - (8 if kind == "e4m3" else 6) - up
        x = torch.stack([codes, -codes]).mul(2.0 ** e).to(dtype)[None]
        y = torch.full((2, 2, 128), big, dtype=dtype)
        check(kind, dtype, block, [x, y])


@pytest.mark.parametrize("kind,dtype", FORMS, ids=IDS)
def test_runs_that_grow_to_the_largest(cuda_lib, kind, dtype):
    g = torch.Generator("cpu").manual_seed(5)
    big = torch.finfo(dtype).max
    for sizes in ([big / 2, big], [big / 40, big / 3, big], [big, big / 1000, big],
                  [1.0, big / 2.01, big, big]):
        runs = [((torch.rand(n, 2, 128, generator=g) * 2 - 1) * s).to(dtype)
                for n, s in zip((3, 1, 5, 2), sizes)]
        for x, s in zip(runs, sizes):
            x[0, :, 9] = s
        check(kind, dtype, 16, runs)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_attention_over_them(cuda_lib, kind):
    """The weights of one token add up to 1: values that are finite give a finite o."""
    first = quant64.TOP[kind] * 2.0 ** (7 if kind == "e4m3" else 9)
    x = torch.full((1, 2, 128), first, dtype=F16)
    y = torch.full((1, 2, 128), torch.finfo(F16).max, dtype=F16)
    cache, (_, v) = stored(kind, F16, 16, [x, y])
    i = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    mask = mab.Mask(kind=mab.ATTN_MASK_NONE, cu_seqlens_q=i([0, 1]), seqlen_k=i([2]), total_q=1,
                    max_seqlen_q=1, max_seqlen_k=2)
    o, lse = mab.paged_fwd(torch.zeros(1, 4, 128, dtype=F16).cuda(), cache, i([[1]]), None, mask,
                           1.0)
    # weights of one half each: the mean of two numbers of 11 bits, rounded once to f16, and
    # the sum of two fp32 products
    want = v.double().mean(0).repeat_interleave(2, 0)[None]
    assert bool(torch.isfinite(o).all())
    assert bool(((o.double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -20)).all())
    assert bool(((lse.double() - math.log(2.0)).abs() <= 2.0 ** -20).all())
