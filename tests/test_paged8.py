"""Argument checks of the 8-bit cache's calls (no GPU): every C call below is
refused on the host, so the fake device addresses are never dereferenced."""
import pytest
import torch

import quant64
from masked_attention_backward_gb300 import binding as mab

FAKE, OFF2, OFF8 = 0x7F0000000000, 0x7F0000000002, 0x7F0000000008
BAD, UNSUP = mab.ATTN_ERR_INVALID_ARG, mab.ATTN_ERR_UNSUPPORTED


def pages(**over):
    a = dict(num_pages=100, page_size=64, Hkv=2, dtype=mab.ATTN_F16, code=mab.ATTN_E4M3, block=16,
             page_stride=16384, head_stride=8192, token_stride=128, scale_page_stride=8,
             scale_head_stride=4)
    a.update(over)
    return mab.attn_pages8_t(**a)


BAD_PAGES = [(dict(num_pages=0), BAD), (dict(num_pages=2 ** 25), BAD), (dict(page_size=0), BAD),
             (dict(page_size=72), UNSUP), (dict(page_size=65552), BAD), (dict(Hkv=0), BAD),
             (dict(Hkv=65536), BAD), (dict(dtype=2), BAD), (dict(code=2), BAD),
             (dict(code=-1), BAD), (dict(block=8), UNSUP), (dict(block=0), UNSUP),
             (dict(block=128), UNSUP), (dict(page_size=48, block=32), BAD),
             (dict(page_stride=0), BAD), (dict(head_stride=136), BAD),
             (dict(token_stride=-128), BAD), (dict(page_stride=2 ** 40), BAD),
             (dict(scale_page_stride=3), BAD), (dict(scale_head_stride=0), BAD),
             (dict(scale_page_stride=2 ** 40), BAD),
             (dict(block=1, scale_page_stride=128, scale_head_stride=72), BAD)]


def _store(pg, T=3, k=FAKE, v=FAKE, ks=256, vs=256, slots=FAKE, kp=FAKE, vp=FAKE, sk=FAKE,
           sv=FAKE):
    return mab.attn_paged8_store(pg, T, k, v, ks, vs, slots, kp, vp, sk, sv, None)


def _load(pg, B=2, total=9, start=FAKE, cu=FAKE, table=FAKE, stride=8, cols=8, kp=FAKE, vp=FAKE,
          sk=FAKE, sv=FAKE, k=FAKE, v=FAKE):
    return mab.attn_paged8_load(pg, B, total, start, cu, table, stride, cols, kp, vp, sk, sv, k, v,
                                None)


@pytest.mark.parametrize("over,want", BAD_PAGES)
def test_page_refusals(over, want):
    assert _store(pages(**over)) == want
    assert _load(pages(**over)) == want


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(T=2 ** 30), dict(k=None), dict(v=None), dict(k=OFF8), dict(v=OFF8),
    dict(ks=128), dict(vs=260), dict(slots=None), dict(slots=FAKE + 4), dict(kp=None),
    dict(vp=OFF8), dict(sk=None), dict(sv=None)])
def test_store_refusals(over):
    assert _store(pages(), **over) == BAD


def test_scales_of_single_tokens_are_aligned():
    one = pages(block=1, scale_page_stride=128, scale_head_stride=64)
    assert _store(one, sk=OFF8) == BAD and _load(one, sv=OFF8) == BAD


@pytest.mark.parametrize("over", [
    dict(B=0), dict(B=65537), dict(total=-1), dict(start=OFF2), dict(cu=None), dict(cu=OFF2),
    dict(table=None), dict(table=OFF2), dict(stride=7), dict(cols=0), dict(cols=2 ** 25,
                                                                          stride=2 ** 25),
    dict(kp=OFF8), dict(vp=None), dict(sk=None), dict(k=None), dict(v=OFF8)])
def test_load_refusals(over):
    assert _load(pages(), **over) == BAD


def test_no_rows_is_no_work():
    assert _store(pages(), T=0) == mab.ATTN_OK and _load(pages(), total=0) == mab.ATTN_OK


def test_cache_handle_checks_its_tensors():
    c = torch.zeros(4, 2, 32, 128, dtype=torch.int8)
    s = torch.zeros(4, 2, 2, dtype=torch.uint8)
    ok = mab.PagedCache8(c, c.clone(), s, s.clone(), torch.float16)
    assert (ok.num_pages, ok.Hkv, ok.page_size, ok.block, ok.dtype) == (4, 2, 32, 16,
                                                                       torch.float16)
    nhd = mab.PagedCache8(c.transpose(1, 2).contiguous(), c.transpose(1, 2).contiguous(), s, s,
                          layout="NHD")
    assert (nhd.Hkv, nhd.page_size) == (2, 32) and nhd.desc.token_stride == 256
    both = torch.zeros(4, 2, 3, 16, 128, dtype=torch.float8_e4m3fn)
    sb = torch.zeros(4, 2, 3, 16, dtype=torch.uint8)
    cut = mab.PagedCache8(both[:, 0], both[:, 1], sb[:, 0], sb[:, 1])
    assert cut.desc.page_stride == 2 * 3 * 16 * 128 and cut.block == 1
    assert (cut.desc.scale_page_stride, cut.desc.scale_head_stride) == (96, 16)
    one = mab.PagedCache8(c[:1, :1], c[:1, :1], s[:1, :1], s[:1, :1])
    assert one.desc.page_stride == 128 and one.desc.scale_page_stride == 2
    e = mab.PagedCache8.empty(3, 2, 64, block=64, codes=torch.int8, layout="NHD", device="cpu")
    assert e.block == 64 and e.k_pages.shape == (3, 64, 2, 128) and e.k_scales.shape == (3, 2, 1)
    for bad in [(c, c[:3], s, s), (c[..., :64], c[..., :64], s, s), (c, c, s, s[:3]),
                (c, c, s.int(), s.int()), (c, c, s[..., :0], s[..., :0]),
                (c, c, torch.zeros(4, 2, 3, dtype=torch.uint8), torch.zeros(4, 2, 3).byte()),
                (c, c, s, torch.zeros(2, 4, 2, dtype=torch.uint8).transpose(0, 1)),
                (c, c.transpose(1, 2).contiguous().transpose(1, 2), s, s),
                (c, c.view(torch.float8_e4m3fn), s, s), (c[0], c[0], s, s)]:
        with pytest.raises(ValueError):
            mab.PagedCache8(*bad)
    with pytest.raises(ValueError):
        mab.PagedCache8(c, c, s, s, layout="DNH")
    with pytest.raises(ValueError):
        mab.PagedCache8.empty(3, 2, 48, block=32, device="cpu")
    for bad in [(c.half(), c.half(), s, s), (c, c, s, s, torch.float32)]:
        with pytest.raises(TypeError):
            mab.PagedCache8(*bad)


def test_binding_refuses_before_the_library():
    c = torch.zeros(4, 2, 32, 128, dtype=torch.int8)
    s = torch.zeros(4, 2, 2, dtype=torch.uint8)
    cache = mab.PagedCache8(c, c, s, s, torch.float16)
    k, slots = torch.zeros(5, 2, 128, dtype=torch.float16), torch.zeros(5, dtype=torch.int64)
    for a in [(k.bfloat16(), k, slots), (k, k[:4], slots), (k, k, slots.int()),
              (k, k.transpose(0, 1).contiguous().transpose(0, 1), slots), (k, k, slots)]:
        with pytest.raises(ValueError):
            mab.paged_store(cache, *a)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)
    for a, kw in [((i(3, 4), i(3), 5), {}), ((i(3, 4).long(), i(4), 5), {}),
                  ((i(4, 3).t(), i(4), 5), {}), ((i(3, 4), i(4).long(), 5), {}),
                  ((i(3, 4), i(4), 5), dict(start=i(2))),
                  ((i(3, 4), i(4), 5), dict(out=(k, k[:4]))),
                  ((i(3, 4), i(4), 5), dict(out=(k, k.bfloat16()))), ((i(3, 4), i(4), 5), {})]:
        with pytest.raises(ValueError):
            mab.paged_load(cache, *a, **kw)
    with pytest.raises(TypeError):
        mab.paged_load(mab.PagedCache(k[:4, :, None].expand(4, 2, 16, 128).contiguous(),
                                      k[:4, :, None].expand(4, 2, 16, 128).contiguous()),
                       i(3, 4), i(4), 5)


def test_plain_form_against_the_types():
    """quant64's codes are torch's: every e4m3 number, and roundings between them."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(codes.double(), quant64.e4m3_numbers())
    x = torch.linspace(-448, 448, 20001, dtype=torch.float64).float()
    x = torch.cat([x, x / 1000, x / 30000])
    want = x.to(torch.float8_e4m3fn).double()
    assert torch.equal(quant64.nearest("e4m3", x.double(), 448.0), want)
    a = torch.tensor([0.0, 448.0, 448.0001, 449.0, 224.0, 1.75, 1.8, 1e-9, 65504.0])
    assert quant64.exponent("e4m3", torch.bfloat16, a.double()).tolist() == \
        [-110, 0, 1, 1, -1, -8, -7, -38, 8]
    assert quant64.exponent("i8", torch.float16, a.double()).tolist() == \
        [-24, 2, 2, 2, 1, -6, -6, -24, 10]
