"""Argument checks of the paged-cache calls (no GPU): every call below is
refused on the host, so the fake device addresses are never dereferenced."""
import pytest
import torch

from masked_attention_backward_gb300 import binding as mab

FAKE, OFF2, OFF8 = 0x7F0000000000, 0x7F0000000002, 0x7F0000000008


def _plan(**over):
    a = dict(B=4, page_size=16, num_pages=100, max_pages=10, table_stride=10, max_tokens=32)
    a.update({n: FAKE for n in ("cached", "fresh", "free_pages", "free_count", "block_table",
                                "cu_seqlens_q", "seqlen_k", "free_count_out", "slot_map",
                                "position", "refused")})
    a.update(over)
    return mab.attn_plan_t(**a)


@pytest.mark.parametrize("over,want", [
    (dict(B=0), mab.ATTN_ERR_INVALID_ARG), (dict(B=4097), mab.ATTN_ERR_INVALID_ARG),
    (dict(page_size=0), mab.ATTN_ERR_INVALID_ARG), (dict(page_size=24), mab.ATTN_ERR_UNSUPPORTED),
    (dict(page_size=65552), mab.ATTN_ERR_INVALID_ARG),
    (dict(num_pages=0), mab.ATTN_ERR_INVALID_ARG),
    (dict(num_pages=2 ** 27), mab.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=2 ** 27, table_stride=2 ** 27), mab.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=0), mab.ATTN_ERR_INVALID_ARG), (dict(table_stride=9), mab.ATTN_ERR_INVALID_ARG),
    (dict(max_tokens=-1), mab.ATTN_ERR_INVALID_ARG),
    (dict(cached=None), mab.ATTN_ERR_INVALID_ARG), (dict(refused=None), mab.ATTN_ERR_INVALID_ARG),
    (dict(fresh=OFF2), mab.ATTN_ERR_INVALID_ARG), (dict(slot_map=None), mab.ATTN_ERR_INVALID_ARG),
    (dict(slot_map=FAKE + 4), mab.ATTN_ERR_INVALID_ARG),
    (dict(position=OFF2), mab.ATTN_ERR_INVALID_ARG),
])
def test_plan_refusals(over, want):
    assert mab.attn_paged_plan(_plan(**over), None) == want


def _pages(**over):
    a = dict(num_pages=100, page_size=16, Hkv=2, dtype=mab.ATTN_F16, page_stride=4096,
             head_stride=2048, token_stride=128)
    a.update(over)
    return mab.attn_pages_t(**a)


def _store(pages, T=3, k=FAKE, v=FAKE, ks=256, vs=256, slots=FAKE, kp=FAKE, vp=FAKE):
    return mab.attn_paged_store(pages, T, k, v, ks, vs, slots, kp, vp, None)


BAD_PAGES = [(dict(num_pages=0), mab.ATTN_ERR_INVALID_ARG),
             (dict(num_pages=2 ** 27), mab.ATTN_ERR_INVALID_ARG),
             (dict(page_size=-16), mab.ATTN_ERR_INVALID_ARG),
             (dict(page_size=40), mab.ATTN_ERR_UNSUPPORTED),
             (dict(Hkv=0), mab.ATTN_ERR_INVALID_ARG), (dict(dtype=2), mab.ATTN_ERR_INVALID_ARG),
             (dict(page_stride=0), mab.ATTN_ERR_INVALID_ARG),
             (dict(head_stride=132), mab.ATTN_ERR_INVALID_ARG),
             (dict(token_stride=-128), mab.ATTN_ERR_INVALID_ARG),
             (dict(page_stride=2 ** 39), mab.ATTN_ERR_INVALID_ARG)]


@pytest.mark.parametrize("over,want", BAD_PAGES)
def test_store_page_refusals(over, want):
    assert _store(_pages(**over)) == want


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(T=2 ** 30), dict(k=None), dict(v=None), dict(k=OFF8), dict(v=OFF8),
    dict(ks=128), dict(vs=260), dict(slots=None), dict(slots=FAKE + 4), dict(kp=None),
    dict(vp=OFF8)])
def test_store_refusals(over):
    assert _store(_pages(), **over) == mab.ATTN_ERR_INVALID_ARG


def test_no_tokens_is_no_work():
    assert _store(_pages(), T=0) == mab.ATTN_OK


def test_cache_handle_checks_its_tensors():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    ok = mab.PagedCache(k, k.clone())
    assert (ok.num_pages, ok.Hkv, ok.page_size) == (4, 2, 16)
    nhd = mab.PagedCache(k, k.clone(), "NHD")
    assert (nhd.Hkv, nhd.page_size) == (16, 2)
    both = torch.zeros(4, 2, 3, 16, 128, dtype=torch.bfloat16)
    cut = mab.PagedCache(both[:, 0], both[:, 1])
    assert cut.desc.page_stride == 2 * 3 * 16 * 128 and cut.desc.head_stride == 16 * 128
    one = mab.PagedCache(k[:1, :1], k[:1, :1])   # strides of single pages and heads say nothing
    assert one.desc.page_stride == 128 and one.desc.token_stride == 128
    for bad in [(k, k.bfloat16()), (k, k[:3]), (k, k.transpose(1, 2).contiguous().transpose(1, 2)),
                (k[..., :64], k[..., :64]), (k[0], k[0]),
                (k.transpose(2, 3), k.transpose(2, 3))]:
        with pytest.raises(ValueError):
            mab.PagedCache(*bad)
    with pytest.raises(ValueError):
        mab.PagedCache(k, k, "DNH")
    with pytest.raises(TypeError):
        mab.PagedCache(k.float(), k.float())


def test_binding_refuses_before_the_library():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    ok = dict(cached=i(3), fresh=i(3), free_pages=i(9), free_count=i(1), block_table=i(3, 4),
              page_size=16, max_tokens=5)
    for over in [dict(fresh=i(2)), dict(cached=i(3).long()), dict(free_count=i(2)),
                 dict(block_table=i(2, 4)), dict(block_table=i(4, 3).t()),
                 dict(cached=i(6)[::2]), dict(out=mab.PagedPlan.empty(2, 5, "cpu")),
                 dict(out=mab.PagedPlan.empty(3, 4, "cpu")), {}]:   # {}: tensors of the host
        with pytest.raises(ValueError):
            mab.paged_plan(**{**ok, **over})
    kp = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    cache = mab.PagedCache(kp, kp)
    k, slots = torch.zeros(5, 2, 128, dtype=torch.float16), torch.zeros(5, dtype=torch.int64)
    for a in [(k.bfloat16(), k, slots), (k, k[:4], slots), (k, k, slots.int()),
              (k, k.transpose(0, 1).contiguous().transpose(0, 1), slots), (k, k, slots)]:
        with pytest.raises(ValueError):
            mab.paged_store(cache, *a)


def _shape(**over):
    a = dict(B=2, Hq=4, Hkv=2, Sq=8, Skv=100, D=128, dtype=mab.ATTN_F16, flags=0)
    a.update(over)
    return mab.attn_shape_t(**a)


SHAPES = [(dict(), mab.ATTN_OK), (dict(B=0), mab.ATTN_ERR_INVALID_ARG),
          (dict(B=4097), mab.ATTN_ERR_INVALID_ARG), (dict(Hq=5), mab.ATTN_ERR_INVALID_ARG),
          (dict(Sq=0), mab.ATTN_ERR_INVALID_ARG), (dict(Skv=2 ** 24 + 1), mab.ATTN_ERR_INVALID_ARG),
          (dict(dtype=3), mab.ATTN_ERR_INVALID_ARG), (dict(flags=1), mab.ATTN_ERR_INVALID_ARG),
          (dict(D=64), mab.ATTN_ERR_UNSUPPORTED), (dict(Hq=129, Hkv=1), mab.ATTN_ERR_UNSUPPORTED),
          (dict(Hq=128, Hkv=1), mab.ATTN_OK)]


@pytest.mark.parametrize("over,want", SHAPES)
def test_paged_workspace_size(over, want):
    assert mab.attn_paged_workspace_size(_shape(**over))[0] == want


def test_workspace_does_not_grow_with_the_lengths():
    n = mab.attn_paged_workspace_size(_shape(Sq=128))[1]
    assert mab.attn_paged_workspace_size(_shape(B=4096, Sq=2 ** 24, Skv=2 ** 24))[1] == n
    assert mab.attn_paged_workspace_size(_shape(Sq=1))[1] < n < 2 ** 25


def _mask(**over):
    a = dict(kind=mab.ATTN_MASK_CAUSAL, window=0, bx=1, by=1, block_mask=None, seqlen_q=None,
             seqlen_k=FAKE, cu_seqlens_q=FAKE, cu_seqlens_k=None, total_q=9, total_k=0, first=0)
    a.update(over)
    return mab.attn_mask_desc_t(**a)


def _fwd(shape=None, pages=None, mask=None, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, stride=8, cols=8,
         sink=None, scale=0.1, o=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 30):
    return mab.attn_paged_fwd(shape or _shape(), pages or _pages(), q, kp, vp, table, stride, cols,
                              sink, mask or _mask(), scale, o, lse, ws, nbytes, None)


@pytest.mark.parametrize("over,want", [x for x in SHAPES if x[1] != mab.ATTN_OK])
def test_fwd_shape_refusals(over, want):
    assert _fwd(shape=_shape(**over)) == want


@pytest.mark.parametrize("over,want", BAD_PAGES)
def test_fwd_page_refusals(over, want):
    assert _fwd(pages=_pages(**over)) == want


@pytest.mark.parametrize("over,want", [
    (dict(pages=_pages(dtype=mab.ATTN_BF16)), mab.ATTN_ERR_INVALID_ARG),
    (dict(pages=_pages(Hkv=4)), mab.ATTN_ERR_INVALID_ARG),
    (dict(scale=0.0), mab.ATTN_ERR_INVALID_ARG), (dict(scale=-1.0), mab.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("nan")), mab.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), mab.ATTN_ERR_INVALID_ARG),
    (dict(cols=0), mab.ATTN_ERR_INVALID_ARG), (dict(stride=7), mab.ATTN_ERR_INVALID_ARG),
    (dict(cols=2 ** 27, stride=2 ** 27), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(kind=mab.ATTN_MASK_BLOCK, block_mask=FAKE)), mab.ATTN_ERR_UNSUPPORTED),
    (dict(mask=_mask(kind=9)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(kind=mab.ATTN_MASK_SLIDING)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(kind=mab.ATTN_MASK_SLIDING_FIRST, window=4, first=-1)),
     mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(kind=mab.ATTN_MASK_SLIDING_FIRST, first=1)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(seqlen_k=None)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(cu_seqlens_q=None)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(seqlen_q=FAKE)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(cu_seqlens_k=FAKE)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(seqlen_k=OFF2)), mab.ATTN_ERR_INVALID_ARG),
    (dict(mask=_mask(total_q=-1)), mab.ATTN_ERR_INVALID_ARG),
    (dict(q=None), mab.ATTN_ERR_INVALID_ARG), (dict(q=OFF8), mab.ATTN_ERR_INVALID_ARG),
    (dict(kp=None), mab.ATTN_ERR_INVALID_ARG), (dict(vp=OFF8), mab.ATTN_ERR_INVALID_ARG),
    (dict(table=None), mab.ATTN_ERR_INVALID_ARG), (dict(table=OFF2), mab.ATTN_ERR_INVALID_ARG),
    (dict(o=None), mab.ATTN_ERR_INVALID_ARG), (dict(lse=OFF2), mab.ATTN_ERR_INVALID_ARG),
    (dict(sink=OFF2), mab.ATTN_ERR_INVALID_ARG), (dict(ws=None), mab.ATTN_ERR_INVALID_ARG),
    (dict(ws=FAKE + 16), mab.ATTN_ERR_INVALID_ARG), (dict(nbytes=1024), mab.ATTN_ERR_WORKSPACE)])
def test_fwd_refusals(over, want):
    assert _fwd(**over) == want


def test_paged_fwd_binding_refusals():
    kp = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    cache = mab.PagedCache(kp, kp)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    q = torch.zeros(5, 4, 128, dtype=torch.float16)
    mask = lambda **kw: mab.Mask(**{**dict(kind=1, cu_seqlens_q=i(4), seqlen_k=i(3), total_q=5,
                                           max_seqlen_q=5, max_seqlen_k=60), **kw})
    ok = dict(q=q, cache=cache, block_table=i(3, 4), sink=None, mask=mask(), scale=0.1)
    for over in [dict(mask=mask(seqlen_k=None)), dict(mask=mask(cu_seqlens_q=i(3))),
                 dict(mask=mask(total_q=4)), dict(q=q.bfloat16()), dict(q=q[None]),
                 dict(q=q.transpose(0, 1)), dict(block_table=i(2, 4)),
                 dict(block_table=i(3, 4).long()), dict(sink=torch.zeros(3)),
                 dict(out=(q[:4], None)), dict(out=(q, torch.zeros(5))), {}]:   # {}: host tensors
        with pytest.raises(ValueError):
            mab.paged_fwd(**{**ok, **over})
