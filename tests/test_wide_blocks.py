"""Mask blocks longer than the sequences, up to the largest int."""
import math

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

WIDE = [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 64), (128, 2 ** 31 - 100), (2 ** 30, 2 ** 30)]


@pytest.mark.parametrize("flags", [0, mab.ATTN_FLAG_SINGLE_PASS])
@pytest.mark.parametrize("bx,by", WIDE)
def test_workspace_holds_the_one_block(bx, by, flags):
    # as many blocks as for blocks of the sequences' lengths
    shape = mab.attn_shape_t(2, 4, 2, 300, 500, 128, mab.ATTN_F16, flags)
    need = lambda x, y: mab.attn_workspace_size(
        shape, mab.attn_mask_desc_t(kind=mab.ATTN_MASK_BLOCK, bx=x, by=y))
    assert need(bx, by) == need(min(bx, 300), min(by, 500))
    assert need(bx, by)[0] == mab.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("bx,by", WIDE)
def test_one_block_for_all(cuda_lib, bx, by):
    B, Hq, Hkv, Sq, Skv, scale = 2, 4, 2, 200, 300, 1.0 / math.sqrt(128)
    g = torch.Generator("cpu").manual_seed(3)
    r = lambda h, s: torch.randn(B, h, s, 128, generator=g).half().cuda()
    q, k, v, dO = r(Hq, Sq), r(Hkv, Skv), r(Hkv, Skv), r(Hq, Sq)
    sink = torch.randn(Hq, generator=g).cuda()
    nq, nk = -(-Sq // bx), -(-Skv // by)
    blocks = torch.ones(B, Hq, nq, nk, dtype=torch.uint8)
    blocks[1, 1, 0, 0] = 0
    i, j = torch.arange(Sq) // bx, torch.arange(Skv) // by
    see = lambda h: lambda b: blocks[b, h][i][:, j].bool().cuda()
    mask = mab.Mask(kind=mab.ATTN_MASK_BLOCK, bx=bx, by=by, block_mask=blocks.cuda())
    o, lse = mab.fwd(q, k, v, sink, mask, scale)
    grads = mab.bwd(q, k, v, o, dO, lse, sink, mask, scale)
    torch.cuda.synchronize()
    dk, dv = (torch.zeros(2, B, Hkv, Skv, 128, dtype=torch.float64, device="cuda")
              for _ in range(2))
    for h in range(Hq):   # every head under its own blocks
        one = slice(h, h + 1)
        kv = slice(h // 2, h // 2 + 1)
        ro, rl, ob, lb = attn64.forward(q[:, one], k[:, kv], v[:, kv], see(h), sink[one], scale)
        attn64.check("o", o[:, one], ro, ob)
        attn64.check("lse", lse[:, one], rl, lb)
        ref = attn64.backward(q[:, one], k[:, kv], v[:, kv], o[:, one], dO[:, one], lse[:, one],
                              see(h), sink[one], scale)
        attn64.check("dq", grads[0][:, one], *ref["dq"])
        attn64.check("dsink", grads[3][one], *ref["dsink"])
        for n, sums in (("dk", dk), ("dv", dv)):
            sums[0][:, kv] += ref[n][0]
            sums[1][:, kv] += ref[n][1]
    # (each head's bound holds a rounding of its own, the group's sum has one)
    attn64.check("dk", grads[1], *dk)
    attn64.check("dv", grads[2], *dv)
