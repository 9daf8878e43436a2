"""Argument checks of the rotary calls and their frequencies (no GPU): every C
call below is refused on the host, so the fake device addresses are never
dereferenced."""
import math

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab

FAKE, OFF2, OFF8 = 0x7F0000000000, 0x7F0000000002, 0x7F0000000008
BAD, UNSUP = mab.ATTN_ERR_INVALID_ARG, mab.ATTN_ERR_UNSUPPORTED


def _desc(**over):
    a = dict(rotary_dim=128, interleaved=0, factor=1.0, turns=FAKE)
    a.update(over)
    return mab.attn_rope_desc_t(**a)


def _tensor(**over):
    a = dict(x=FAKE, y=FAKE, heads=4, x_batch=4096, x_head=128, x_token=512, y_batch=4096,
             y_head=128, y_token=512)
    a.update(over)
    return mab.attn_rope_tensor_t(**a)


def _rope(desc=None, dtype=mab.ATTN_BF16, B=2, S=8, q=None, k=None, position=FAKE, stride=8):
    return mab.attn_rope(desc or _desc(), dtype, B, S, q or _tensor(), k, position, stride, 0, None)


@pytest.mark.parametrize("over,want", [
    (dict(rotary_dim=0), BAD), (dict(rotary_dim=-16), BAD), (dict(rotary_dim=31), BAD),
    (dict(rotary_dim=144), BAD), (dict(rotary_dim=24), UNSUP), (dict(rotary_dim=2), UNSUP),
    (dict(turns=None), BAD), (dict(turns=FAKE + 4), BAD), (dict(factor=math.inf), BAD),
    (dict(factor=math.nan), BAD)])
def test_desc_refusals(over, want):
    assert _rope(_desc(**over)) == want


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(B=0), dict(B=65536), dict(S=-1), dict(position=OFF2), dict(stride=-1)])
def test_call_refusals(over):
    assert _rope(**over) == BAD


@pytest.mark.parametrize("over", [
    dict(x=None), dict(y=None), dict(x=OFF8), dict(y=OFF8), dict(heads=0), dict(heads=65536),
    dict(x_head=-128), dict(x_token=132), dict(x_batch=2 ** 40), dict(y_head=0),
    dict(y_token=120), dict(y_batch=2 ** 40), dict(y_token=516)])
def test_tensor_refusals(over):
    assert _rope(q=_tensor(**over)) == BAD
    assert _rope(k=_tensor(**over)) == BAD


def test_no_tokens_is_no_work():
    assert _rope(S=0) == mab.ATTN_OK


def test_binding_refuses_before_the_library():
    rp = mab.Rope(64, device="cpu")
    z = lambda *n, dt=torch.bfloat16: torch.zeros(*n, dtype=dt)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    q, k = z(5, 4, 128), z(5, 2, 128)
    for a in [(z(5, 128), k), (z(5, 4, 64), k), (z(5, 128, 4).transpose(1, 2), k),
              (q, z(4, 2, 128)), (q, z(5, 2, 128, dt=torch.float16)), (q, z(1, 2, 5, 128)),
              (z(2, 4, 5, 128), z(1, 2, 5, 128)), (q, k, i(4)), (q, k, i(5).long()),
              (q, k, i(10)[::2]), (z(2, 4, 5, 128), None, i(1, 5)), (q, k, None, (q, None)),
              (q, None, None, (q, k)), (q, k, None, (q[:, :3], k)),
              (q, k, None, (q.half(), k)), (q, k)]:   # the last: tensors of the host
        with pytest.raises(ValueError):
            mab.rope(rp, *a)
    with pytest.raises(TypeError):
        mab.rope(rp, q.float())


def test_frequencies():
    w, f = mab.rope_frequencies(8, 10000.0)
    assert f == 1.0 and w == [10000.0 ** (-i / 4) for i in range(4)]
    w4, _ = mab.rope_frequencies(8, 10000.0, mab.RopeScaling("linear", 4.0))
    assert all(a == b / 4 for a, b in zip(w4, w))
    wr, _ = mab.rope_frequencies(8, 10000.0, mab.RopeScaling("raised", 4.0))
    assert wr[0] == 1.0 and math.isclose(wr[3], w[3] / 4, rel_tol=1e-12)
    wp, f = mab.rope_frequencies(128, 10000.0, mab.RopeScaling("parts", 8.0, original_length=4096))
    w, _ = mab.rope_frequencies(128, 10000.0)
    assert wp[0] == w[0] and math.isclose(wp[-1], w[-1] / 8, rel_tol=1e-15)
    assert all(b / 8 <= a <= b for a, b in zip(wp, w)) and f == 0.1 * math.log(8) + 1
    assert mab.rope_frequencies(128, scaling=mab.RopeScaling("parts", 8.0, 4096, attention=1.0))[
        1] == 1.0
    for a in [(7,), (0,), (8, -1.0), (8, 1e4, mab.RopeScaling("other", 2.0)),
              (8, 1e4, mab.RopeScaling("linear", 0.0)), (2, 1e4, mab.RopeScaling("raised", 2.0)),
              (8, 1e4, mab.RopeScaling("parts", 2.0)),
              (8, 1e4, mab.RopeScaling("parts", 2.0, 4096, low=4.0, high=4.0))]:
        with pytest.raises(ValueError):
            mab.rope_frequencies(*a)


def test_handle():
    rp = mab.Rope(32, frequencies=[2 * math.pi / 4] * 15 + [-2 * math.pi / 8], device="cpu")
    assert rp.turns[0] == 2 ** 62 and rp.turns[15] == -2 ** 61
    for bad in [dict(frequencies=[1.0]), dict(frequencies=[math.nan] * 16),
                dict(frequencies=[1.0] * 16, scaling=mab.RopeScaling("linear", 2.0))]:
        with pytest.raises(ValueError):
            mab.Rope(32, device="cpu", **bad)
