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
