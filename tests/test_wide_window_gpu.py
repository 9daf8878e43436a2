"""A sliding window longer than the sequence, up to the largest int, is the
causal mask: the same results as a window of the sequence's length."""
import math

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128)
WIDE = [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30]


def _inputs(B, Hq, Hkv, S, seed=0):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).half().cuda()
    return (r(B, Hq, S, 128), r(B, Hkv, S, 128), r(B, Hkv, S, 128), r(B, Hq, S, 128),
            torch.randn(Hq, generator=g).cuda())


def _step(q, k, v, dO, sink, mask, **kw):
    o, lse = mab.fwd(q, k, v, sink, mask, SCALE)
    out = (o, lse) + mab.bwd(q, k, v, o, dO, lse, sink, mask, SCALE, **kw)
    torch.cuda.synchronize()
    return out


def _same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("window", WIDE)
@pytest.mark.parametrize("S", [1, 100, 333, 700])
def test_window_past_the_sequence(cuda_lib, S, window):
    data = _inputs(2, 4, 2, S, S)
    at = lambda w: mab.Mask(kind=mab.ATTN_MASK_SLIDING, window=w)
    got = _step(*data, at(window))
    _same(got, _step(*data, at(S)))
    # against the formula
    q, k, v, dO, sink = data
    i = torch.arange(S, device="cuda")
    ref = attn64.backward(q, k, v, got[0], dO, got[1], lambda b: attn64.window_first(i, i), sink,
                          SCALE)
    for n, x in zip(("dq", "dk", "dv", "dsink"), got[2:]):
        attn64.check(n, x, *ref[n])


@pytest.mark.parametrize("window", WIDE[:2])
@pytest.mark.parametrize("how", ["compensated", "single_pass", "tile", "units"])
def test_every_form_of_the_backward(cuda_lib, monkeypatch, how, window):
    if how in ("tile", "units"):
        monkeypatch.setenv("MASKATTN_DKDV_SCHEDULE", how)
    kw = {how: True} if how in ("compensated", "single_pass") else {}
    data = _inputs(1, 4, 1, 500, 7)
    at = lambda w: mab.Mask(kind=mab.ATTN_MASK_SLIDING, window=w)
    _same(_step(*data, at(window), **kw), _step(*data, at(500), **kw))


@pytest.mark.parametrize("window", WIDE[:2])
def test_lengths(cuda_lib, window):
    S, lens = 300, [300, 1, 129, 0]
    q, k, v, dO, sink = _inputs(4, 2, 1, S, 9)
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    at = lambda w: mab.Mask(kind=mab.ATTN_MASK_SLIDING, window=w, seqlen_q=t, seqlen_k=t)
    _same(_step(q, k, v, dO, sink, at(window)), _step(q, k, v, dO, sink, at(S)))
    pack = lambda x: torch.cat([x[b, :, :n].transpose(0, 1) for b, n in enumerate(lens)]) \
        .contiguous()
    at = lambda w: mab.packed_mask(mab.ATTN_MASK_SLIDING, lens, lens, "cuda", window=w)
    data = [pack(x) for x in (q, k, v, dO)] + [sink]
    _same(_step(*data, at(window)), _step(*data, at(S)))
