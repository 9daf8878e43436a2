"""Argument checks of the sliding window with first keys (no GPU)."""
import pytest

from masked_attention_backward_gb300 import binding as mab


def _shape(Sq=256, Skv=256, flags=0):
    return mab.attn_shape_t(1, 4, 2, Sq, Skv, 128, mab.ATTN_BF16, flags)


def _mask(window=64, first=4):
    return mab.Mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=window, first=first).desc()


@pytest.mark.parametrize("shape,mask,want", [
    (_shape(), _mask(), mab.ATTN_OK),
    (_shape(), _mask(first=0), mab.ATTN_OK),
    (_shape(), _mask(window=2 ** 31 - 1, first=2 ** 31 - 1), mab.ATTN_OK),
    (_shape(), _mask(window=0), mab.ATTN_ERR_INVALID_ARG),
    (_shape(), _mask(window=-5), mab.ATTN_ERR_INVALID_ARG),
    (_shape(), _mask(first=-1), mab.ATTN_ERR_INVALID_ARG),
    (_shape(Sq=255), _mask(), mab.ATTN_ERR_INVALID_ARG),
    (_shape(flags=mab.ATTN_FLAG_COMPENSATED), _mask(), mab.ATTN_OK),
    (_shape(flags=mab.ATTN_FLAG_SINGLE_PASS), _mask(), mab.ATTN_ERR_UNSUPPORTED),
])
def test_workspace_size_validation(shape, mask, want):
    assert mab.attn_workspace_size(shape, mask)[0] == want


def test_first_is_ignored_by_other_kinds():
    for kind in (mab.ATTN_MASK_NONE, mab.ATTN_MASK_CAUSAL, mab.ATTN_MASK_SLIDING):
        r, n = mab.attn_workspace_size(_shape(), mab.Mask(kind=kind, window=9).desc())
        r2, n2 = mab.attn_workspace_size(_shape(), mab.Mask(kind=kind, window=9, first=-3).desc())
        assert r == r2 == mab.ATTN_OK and n == n2
