"""The forward on many units of a few steps each: a softmax group that is done
with a unit must not replace its queries before the other group's last scores."""
import math

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [64, 130, 190])
def test_many_short_units(cuda_lib, S):
    B, Hq, Hkv = 900, 4, 2
    g = torch.Generator("cuda").manual_seed(S)
    r = lambda h: torch.randn(B, h, S, 128, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = r(Hq), r(Hkv), r(Hkv)
    sink = torch.randn(Hq, generator=g, device="cuda")
    for mask in (mab.Mask(kind=mab.ATTN_MASK_NONE), mab.Mask(kind=mab.ATTN_MASK_CAUSAL)):
        i = torch.arange(S, device="cuda")
        vis = attn64.window_first(i, i) if mask.kind == mab.ATTN_MASK_CAUSAL else \
            torch.ones(S, S, dtype=torch.bool, device="cuda")
        o, lse = mab.fwd(q, k, v, sink, mask, 1 / math.sqrt(128))
        torch.cuda.synchronize()
        ro, rl, ob, lb = attn64.forward(q, k, v, lambda b: vis, sink, 1 / math.sqrt(128))
        attn64.check("o", o, ro, ob)
        attn64.check("lse", lse, rl, lb)
