"""Rotary positions against the formula in 64 bits.

Bound of an element y = f (x1 cos - x2 sin): the angle's fraction is rounded to
24 bits (at most pi 2^-24 of an angle below pi), cos and sin are off by an ulp at
most (2^-24 below 1), their products with f and with x and the sum are rounded to
24 bits: together below f (|x1| + |x2|) 2^-21; then one rounding to 16 bits."""
import math

import pytest
import torch

import attn64
from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _angles(rp, pos):
    """Angles below half a turn of the exact product, [.., R / 2] in 64 bits."""
    turns = [int(t) % 2 ** 64 for t in rp.turns.tolist()]
    rows = []
    for x in pos.flatten().tolist():
        f = [(t * x) % 2 ** 64 for t in turns]
        rows.append([(v - 2 ** 64 if v >= 2 ** 63 else v) / 2.0 ** 64 * 2 * math.pi for v in f])
    return torch.tensor(rows, dtype=torch.float64).reshape(*pos.shape, len(turns)).cuda()


def _plain(rp, x, angle, inverse):
    """x [.., 128] under angle [.., R / 2] (broadcast over heads): value, bound."""
    R, x = rp.rotary_dim, x.double()
    f = rp.factor
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if rp.interleaved else (x[..., :R // 2], x[..., R // 2:R])
    s = -torch.sin(angle) if inverse else torch.sin(angle)
    c = torch.cos(angle)
    y1, y2 = f * (a * c - b * s), f * (b * c + a * s)
    e = abs(f) * (a.abs() + b.abs()) * 2.0 ** -21
    join = (lambda u, v: torch.stack([u, v], -1).flatten(-2)) if rp.interleaved else \
        (lambda u, v: torch.cat([u, v], -1))
    y = torch.cat([join(y1, y2), x[..., R:]], -1)
    return y, torch.cat([join(e, e), torch.zeros_like(x[..., R:])], -1)


def _check(name, got, rp, x, angle, inverse):
    y, e = _plain(rp, x, angle, inverse)
    u, tiny = attn64.u_of(x.dtype), attn64.tiny_of(x.dtype)
    R = rp.rotary_dim
    attn64.check(name, got[..., :R], y[..., :R], e[..., :R] + u * y[..., :R].abs() + tiny)
    assert torch.equal(got[..., R:], x[..., R:]), name


def _randn(seed, *shape, dtype):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [16, 48, 64, 112, 128])
def test_rows(cuda_lib, R, interleaved, dtype):
    T = 37
    qkv = _randn(R, T, 5 + 3 + 3, 128, dtype=dtype)
    q, k = qkv[:, :5], qkv[:, 5:8]     # slices of a projection's output
    rp = mab.Rope(R, 10000.0, interleaved, mab.RopeScaling("parts", 8.0, original_length=4096))
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(R),
                        dtype=torch.int32)
    before = qkv.clone()
    for inverse, turn in ((False, mab.rope), (True, mab.rope_bwd)):
        y, z = turn(rp, q, k, pos.cuda())
        ang = _angles(rp, pos)[:, None]
        _check("q", y, rp, q, ang, inverse)
        _check("k", z, rp, k, ang, inverse)
    assert torch.equal(qkv, before)


@pytest.mark.parametrize("B,Hq,Hkv,S", [(1, 1, 1, 1), (2, 3, 1, 17), (3, 8, 2, 130), (1, 33, 5, 16)])
@pytest.mark.parametrize("how", ["counted", "shared", "own"])
def test_heads(cuda_lib, B, Hq, Hkv, S, how):
    rp = mab.Rope(128, 500000.0)
    q, k = _randn(S, B, Hq, S, 128, dtype=BF16), _randn(S + 1, B, Hkv, S, 128, dtype=BF16)
    g = torch.Generator().manual_seed(S)
    pos = {"counted": None, "shared": torch.randint(0, 9999, (S,), generator=g, dtype=torch.int32),
           "own": torch.randint(0, 9999, (B, S), generator=g, dtype=torch.int32)}[how]
    y, z = mab.rope(rp, q, k, None if pos is None else pos.cuda())
    full = torch.arange(S) if pos is None else pos
    ang = _angles(rp, full.expand(B, S) if full.dim() == 1 else full)[:, None]
    _check("q", y, rp, q, ang, False)
    _check("k", z, rp, k, ang, False)
    alone, none = mab.rope(rp, q, None, None if pos is None else pos.cuda())
    assert none is None and torch.equal(alone, y)


@pytest.mark.parametrize("pos", [0, 1, 2 ** 24 - 1, 2 ** 24 + 1, 2 ** 31 - 1])
def test_far_positions(cuda_lib, pos):
    """Angles of the largest positions are as exact as those of the first."""
    rp = mab.Rope(128)
    q = _randn(1, 3, 2, 128, dtype=F16)
    p = torch.full((3,), pos, dtype=torch.int32)
    y, _ = mab.rope(rp, q, None, p.cuda())
    _check("q", y, rp, q, _angles(rp, p)[:, None], False)
    if pos == 0:
        assert torch.equal(y, q)


def test_padding_rows_and_in_place(cuda_lib):
    rp = mab.Rope(64, interleaved=True)
    q, k = _randn(2, 9, 4, 128, dtype=BF16), _randn(3, 9, 2, 128, dtype=BF16)
    pos = torch.tensor([5, 0, -1, 7, 100, -2 ** 31, 3, 2, -1], dtype=torch.int32).cuda()
    out = (torch.full_like(q, 7.0), torch.full_like(k, 7.0))
    mab.rope(rp, q, k, pos, out=out)
    live = pos >= 0
    for o, x in zip(out, (q, k)):
        assert bool((o[~live] == 7).all())
        _check("rows", o[live], rp, x[live], _angles(rp, pos[live].cpu())[:, None], False)
    here = (q.clone(), k.clone())
    mab.rope(rp, *here, pos, out=here)
    for h, o, x in zip(here, out, (q, k)):
        assert torch.equal(h[live], o[live]) and torch.equal(h[~live], x[~live])


def test_broadcast_and_transposed_inputs(cuda_lib):
    """One head for all (stride 0), and [B, S, H, 128] read as [B, H, S, 128]."""
    rp = mab.Rope(128)
    one = _randn(4, 2, 1, 20, 128, dtype=F16)
    q = one.expand(2, 6, 20, 128)
    k = _randn(5, 2, 20, 3, 128, dtype=F16).transpose(1, 2)
    y, z = mab.rope(rp, q, k)
    ang = _angles(rp, torch.arange(20).expand(2, 20))[:, None]
    _check("q", y, rp, q, ang, False)
    _check("k", z, rp, k, ang, False)
    to = torch.empty(2, 20, 3, 128, dtype=F16, device="cuda").transpose(1, 2)
    mab.rope(rp, k, None, out=(to, None))
    assert torch.equal(to, z)


def test_gradient_by_differences(cuda_lib):
    """rope is linear: <rope(x), g> = <x, rope_bwd(g)>, and so for differences."""
    rp = mab.Rope(96, scaling=mab.RopeScaling("raised", 4.0))
    x, d, g = (_randn(s, 1, 4, 33, 128, dtype=F16) for s in (6, 7, 8))
    gx, _ = mab.rope_bwd(rp, g)
    y0, y1 = (mab.rope(rp, v)[0] for v in (x, (x + d)))
    moved = (x + d).double() - x.double()
    left = ((y1.double() - y0.double()) * g.double()).sum()
    right = (moved * gx.double()).sum()
    ang = _angles(rp, torch.arange(33).expand(1, 33))[:, None]

    def off(v, inverse):   # how far each element of the call's result may be off
        y, e = _plain(rp, v, ang, inverse)
        return e + 2.0 ** -11 * y.abs() + attn64.tiny_of(F16)
    bound = (g.double().abs() * (off(x, False) + off(x + d, False))).sum() + \
        (moved.abs() * off(g, True)).sum()
    assert (left - right).abs() <= bound


def test_special_values(cuda_lib):
    """What is not finite stays in its pair."""
    rp = mab.Rope(32)
    q = _randn(9, 4, 2, 128, dtype=BF16)
    q[1, 0, 3] = float("inf")
    q[2, 1, 20] = float("nan")
    q[3, 0, 100] = float("-inf")     # not turned
    y, _ = mab.rope(rp, q, None, torch.tensor([3, 3, 3, 3], dtype=torch.int32).cuda())
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 19] = want[2, 1, 4] = want[2, 1, 20] = want[3, 0, 100] = True
    assert torch.equal(bad, want)


def test_captured(cuda_lib):
    """Replayed with other positions and rows."""
    rp = mab.Rope(128)
    q, k = _randn(10, 6, 4, 128, dtype=BF16), _randn(11, 6, 2, 128, dtype=BF16)
    pos = torch.arange(6, dtype=torch.int32).cuda()
    out = (torch.empty_like(q), torch.empty_like(k))
    mab.rope(rp, q, k, pos, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mab.rope(rp, q, k, pos, out=out)
    q.copy_(_randn(12, 6, 4, 128, dtype=BF16))
    pos.add_(1000)
    g.replay()
    ang = _angles(rp, pos.cpu())[:, None]
    _check("q", out[0], rp, q, ang, False)
    _check("k", out[1], rp, k, ang, False)
