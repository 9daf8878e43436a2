"""Query rows that are not finite, in both forwards: what such a row gives, and
that no other row changes."""
import math

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SCALE = 1.0 / math.sqrt(128)
S = 128


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _short_units(form, n):
    """n sequences whose units have two steps or more, then n whose units have
    one (of which the second group of softmax warps has none): the mask, the
    shape of q, that of k, and the rows of q that are in the problem."""
    if form == "padded":
        mask = mab.Mask(kind=mab.ATTN_MASK_NONE, seqlen_k=_i32([128] * n + [64] * n))
        return mask, (2 * n, 1, S, 128), (2 * n, 1, S, 128)
    if form == "packed":
        mask = mab.packed_mask(mab.ATTN_MASK_NONE, [S] * (2 * n), [128] * n + [50] * n, "cuda")
        return mask, (2 * n * S, 1, 128), (n * 178, 1, 128)
    # every key block, or one of them
    blocks = torch.ones(2 * n, 1, 1, 4, dtype=torch.uint8)
    blocks[n:] = 0
    blocks[n:, :, :, 2] = 1
    mask = mab.Mask(kind=mab.ATTN_MASK_BLOCK, bx=128, by=64, block_mask=blocks.cuda())
    return mask, (2 * n, 1, S, 128), (2 * n, 1, 256, 128)


@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("form", ["padded", "packed", "block"])
def test_units_of_one_step_keep_their_other_rows(cuda_lib, form, sink):
    # the first sequences leave NaN in row 5 of an accumulator that the later
    # ones, each with a NaN row of its own beside row 5, do not write
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    mask, qs, ks = _short_units(form, n)
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda s: torch.randn(s, generator=g, device="cuda").to(F16)
    q, k, v = r(qs), r(ks), r(ks)
    sk = torch.ones(1, device="cuda") if sink else None
    want, want_lse = mab.fwd(q, k, v, sk, mask, SCALE)
    bad = q.clone()
    rows = bad.view(2 * n, S, 128)
    rows[:n, 5, 3] = float("nan")
    rows[n:, 7, 3] = float("nan")
    o, lse = mab.fwd(bad, k, v, sk, mask, SCALE)
    torch.cuda.synchronize()
    o, lse, want, want_lse = o.view(2 * n, S, 128), lse.view(2 * n, S), want.view(2 * n, S, 128), \
        want_lse.view(2 * n, S)
    for part, row in ((slice(0, n), 5), (slice(n, 2 * n), 7)):
        assert bool(o[part, row].isnan().all()) and bool(lse[part, row].isnan().all())
        o[part, row], lse[part, row] = want[part, row], want_lse[part, row]
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("L", [1, 40, 64])
def test_short_sequences_after_long_ones(cuda_lib, L):
    # the same from one call to the next
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator("cuda").manual_seed(L)
    r = lambda s: torch.randn(n, 1, s, 128, generator=g, device="cuda").to(BF16)
    none, causal = mab.Mask(kind=mab.ATTN_MASK_NONE), mab.Mask(kind=mab.ATTN_MASK_CAUSAL)
    before = r(128).fill_(float("nan"))
    q, k, v = r(L), r(L), r(L)
    want, want_lse = mab.fwd(q, k, v, None, causal, SCALE)
    q[:, :, L - 1, 9] = float("nan")
    mab.fwd(before, r(128), r(128), None, none, SCALE)
    o, lse = mab.fwd(q, k, v, None, causal, SCALE)
    torch.cuda.synchronize()
    assert bool(o[:, :, L - 1].isnan().all()) and bool(lse[:, :, L - 1].isnan().all())
    assert torch.equal(o[:, :, :L - 1], want[:, :, :L - 1])
    assert torch.equal(lse[:, :, :L - 1], want_lse[:, :, :L - 1])


# An infinite element of a query against keys that are all of one sign there:
# logits of +inf alone (inf - inf: NaN) or of -inf alone (they weigh nothing).
@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("keys", [1, 2, 63, 64, 130])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_query_over_keys_of_one_sign(cuda_lib, sign, keys, sink):
    g = torch.Generator("cuda").manual_seed(keys)
    r = lambda h: torch.randn(1, h, keys, 128, generator=g, device="cuda").to(F16)
    q, k, v = r(4), r(2), r(2)
    k[..., 5] = k[..., 5].abs() + 0.1
    sk = torch.tensor([0.5, -0.5, 1.0, -1.0], device="cuda") if sink else None
    want, want_lse = mab.fwd(q, k, v, sk, mab.Mask(kind=mab.ATTN_MASK_CAUSAL), SCALE)
    rows = sorted({0, keys // 2, keys - 1})
    bad = q.clone()
    bad[0, 2, rows, 5] = sign * math.inf
    got = {"fwd": mab.fwd(bad, k, v, sk, mab.Mask(kind=mab.ATTN_MASK_CAUSAL), SCALE)}
    # the same keys in pages of 16
    n = -(-keys // 16)
    pages = torch.zeros(2, n, 2, 16, 128, dtype=F16, device="cuda")
    for x, to in zip((k, v), pages):
        flat = torch.zeros(2, 16 * n, 128, dtype=F16, device="cuda")
        flat[:, :keys] = x[0]
        to.copy_(flat.view(2, n, 16, 128).transpose(0, 1))
    mask = mab.Mask(kind=mab.ATTN_MASK_CAUSAL, cu_seqlens_q=_i32([0, keys]), seqlen_k=_i32([keys]),
                    total_q=keys, max_seqlen_q=keys, max_seqlen_k=keys)
    o, lse = mab.paged_fwd(bad[0].transpose(0, 1).contiguous(), mab.PagedCache(*pages),
                           _i32([list(range(n))]), sk, mask, SCALE)
    got["paged_fwd"] = (o.transpose(0, 1)[None], lse)
    torch.cuda.synchronize()
    for name, (o, lse) in got.items():
        o, lse = o[0, 2].float(), lse.reshape(4, keys)[2]
        if sign > 0:
            assert bool(o[rows].isnan().all()) and bool(lse[rows].isnan().all()), name
        else:
            assert bool((o[rows] == 0).all()), name
            # the sink through a change of base and back: two products and their
            # constants, each off by 2^-24
            at = torch.full_like(lse[rows], 1.0 if sink else math.inf)
            assert torch.allclose(lse[rows], at, rtol=2.0 ** -22, atol=0), name
        rest = [i for i in range(keys) if i not in rows]
        assert bool(torch.isfinite(o[rest]).all()) and bool(torch.isfinite(lse[rest]).all()), name
        if name == "fwd":
            assert torch.equal(o[rest], want[0, 2].float()[rest])
            assert torch.equal(lse[rest], want_lse.reshape(4, keys)[2][rest])
