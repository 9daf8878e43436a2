"""Page planning and the cache store against loops over requests and tokens."""
import random

import pytest
import torch

from masked_attention_backward_gb300 import binding as mab

pytestmark = pytest.mark.gpu


def _reference(cached, fresh, stack, count, table, ps, num_pages, max_tokens):
    """The planning rules, one request and one token at a time (lists)."""
    stack, table = list(stack), [list(r) for r in table]
    cols = len(table[0])
    cached = [max(c, 0) for c in cached]
    for b, (c, f) in enumerate(zip(cached, fresh)):
        if f < 0:
            for i in range(min(-(-c // ps), cols)):
                if count < num_pages:
                    stack[count] = table[b][i]
                    count += 1
    end, need_upto, refused, avail = 0, 0, 0, count
    cu, lens, slots, pos = [0], [], [-1] * max_tokens, [-1] * max_tokens
    for b, (c, f) in enumerate(zip(cached, fresh)):
        start, end = end, end + max(f, 0)
        cu.append(min(end, 2 ** 31 - 1))
        if f < 0:
            lens.append(0)
            continue
        ok = c + f <= cols * ps and end <= max_tokens
        if ok:
            held = -(-c // ps)
            need = -(-(c + f) // ps) - held
            need_upto += need
            ok = need == 0 or need_upto <= avail
        if ok:
            for i in range(need):
                count -= 1
                table[b][held + i] = stack[count]
        else:
            refused += 1
        lens.append(c + f if ok else c)
        for t in range(start, min(end, max_tokens)):
            pos[t] = min(c + t - start, 2 ** 31 - 1)
            if ok:
                page = table[b][pos[t] // ps]
                slots[t] = page * ps + pos[t] % ps if 0 <= page < num_pages else -1
    return dict(cu_seqlens_q=cu, seqlen_k=lens, free_count=[count], slot_map=slots, position=pos,
                refused=[refused]), stack, table


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _compare(cached, fresh, stack, count, table, ps, max_tokens, stride=0, alias=False):
    B, cols, P = len(cached), len(table[0]), len(stack)
    ref, rstack, rtable = _reference(cached, fresh, stack, count, table, ps, P, max_tokens)
    wide = torch.full((B, cols + stride), -9, dtype=torch.int32, device="cuda")
    wide[:, :cols] = _i32(table)
    tab, dstack, dc, dn = wide[:, :cols], _i32(stack), _i32(cached), _i32([count])
    out = None
    if alias:
        out = mab.PagedPlan.empty(B, max_tokens, "cuda")
        out.seqlen_k, out.free_count = dc, dn
    plan = mab.paged_plan(dc, _i32(fresh), dstack, dn, tab, ps, max_tokens, out=out)
    torch.cuda.synchronize()
    for n, want in ref.items():
        assert getattr(plan, n).tolist() == want, n
    assert dstack.tolist() == rstack and tab.tolist() == rtable
    assert bool((wide[:, cols:] == -9).all())
    return plan


def _random(seed, B, ps, hi, new, cols_extra=2, spare=5, ended=0.1):
    r = random.Random(seed)
    cached = [r.choice([0, 1, ps, ps - 1, r.randint(0, hi)]) for _ in range(B)]
    fresh = [-1 if r.random() < ended else r.choice([0, 1, ps, r.randint(0, new)])
             for _ in range(B)]
    cols = -(-(max(hi, ps) + max(new, ps)) // ps) + cols_extra
    held = [-(-c // ps) for c in cached]
    need = sum(max(0, -(-(c + f) // ps) - h) for c, f, h in zip(cached, fresh, held) if f >= 0)
    P = max(sum(held) + need + spare, 1)
    ids = list(range(P))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (cols - h))
        at += h
    stack = ids[at:] + [-3] * at
    return cached, fresh, stack, P - at, table


@pytest.mark.parametrize("B,ps,hi,new", [(1, 16, 1, 1), (1, 64, 500, 300), (7, 16, 100, 40),
                                         (33, 48, 2000, 9), (256, 128, 3000, 70),
                                         (1024, 16, 300, 3), (1025, 32, 90, 20),
                                         (4096, 16, 50, 5)])
@pytest.mark.parametrize("alias", [False, True])
def test_plan(cuda_lib, B, ps, hi, new, alias):
    for seed in range(2):
        c, f, s, n, t = _random(B * 10 + seed, B, ps, hi, new)
        T = sum(max(x, 0) for x in f) + seed * 13
        _compare(c, f, s, n, t, ps, T, stride=3 * seed, alias=alias)


def test_plan_long_chunks(cuda_lib):
    # more tokens than one block's threads, several blocks of a cluster
    c, f, s, n, t = _random(5, 9, 64, 4000, 9000)
    _compare(c, f, s, n, t, 64, sum(max(x, 0) for x in f) + 100)


@pytest.mark.parametrize("short", [1, 2, 5, 1000])
def test_pool_that_runs_out(cuda_lib, short):
    c, f, s, n, t = _random(short, 40, 16, 60, 50, spare=0)
    T = sum(max(x, 0) for x in f)
    # the ended requests' pages must not make up for what is missing
    f = [max(x, 0) for x in f]
    plan = _compare(c, f, s, max(n - short, 0), t, 16, T)
    assert int(plan.refused) > 0


def test_too_many_tokens_or_columns(cuda_lib):
    c, f, s, n, t = _random(3, 30, 16, 60, 50, ended=0)
    T = sum(f)
    _compare(c, f, s, n, t, 16, T // 2)
    _compare(c, f, s, n, t, 16, 0)
    _compare(c, f, s, n, [r[:4] for r in t], 16, T)   # rows shorter than some requests
    c, f = c[:6], f[:6]
    c[3], f[5] = 2 ** 31 - 1, 2 ** 31 - 1
    assert int(_compare(c, f, s, n, t[:6], 16, T).refused) >= 2


def test_bad_numbers_stay_in_bounds(cuda_lib):
    c, f, s, n, t = _random(4, 12, 16, 90, 40)
    for row in t:
        for i in range(0, len(row), 2):
            row[i] = [-5, 10 ** 9][i % 4 // 2]
    s = [x if i % 3 else 2 ** 31 - 1 for i, x in enumerate(s)]
    _compare(c, f, s, n, t, 16, sum(max(x, 0) for x in f))
    c = [-x for x in c]
    _compare(c, f, s, n, t, 16, sum(max(x, 0) for x in f))
    ended = [-1] * len(f)   # more pages come back than the stack holds
    _compare([90] * len(f), ended, s, len(s) - 3, t, 16, 4)


def test_repeated_and_captured(cuda_lib):
    c, f, s, n, t = _random(6, 50, 16, 200, 30)
    T = sum(max(x, 0) for x in f) + 5
    ref, rstack, rtable = _reference(c, f, s, n, t, 16, len(s), T)
    dc, df, ds, dn, dt = _i32(c), _i32(f), _i32(s), _i32([n]), _i32(t)
    out = mab.PagedPlan.empty(len(c), T, "cuda")
    mab.paged_plan(dc, df, ds, dn, dt, 16, T, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mab.paged_plan(dc, df, ds, dn, dt, 16, T, out=out)
    for x in (out.cu_seqlens_q, out.seqlen_k, out.slot_map, out.position, out.refused):
        x.fill_(77)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for name, want in ref.items():
        assert getattr(out, name).tolist() == want, name
    assert ds.tolist() == rstack and dt.tolist() == rtable


# ------------------------------------------------------------------ store

def _pages(layout, P, Hkv, ps, dtype, how):
    shape = (P, Hkv, ps, 128) if layout == "HND" else (P, ps, Hkv, 128)
    g = torch.Generator("cuda").manual_seed(P)
    if how == "interleaved":   # K and V side by side in one tensor
        both = torch.randn((P, 2) + shape[1:], generator=g, device="cuda").to(dtype)
        return both[:, 0], both[:, 1]
    k = torch.randn(shape, generator=g, device="cuda").to(dtype)
    return k, k.flip(0).contiguous()


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("how", ["plain", "interleaved"])
@pytest.mark.parametrize("T,P,Hkv,ps", [(1, 1, 1, 16), (3, 2, 3, 16), (33, 9, 8, 48),
                                        (500, 40, 2, 64), (2000, 300, 5, 32)])
def test_store(cuda_lib, layout, how, T, P, Hkv, ps):
    for dtype in (torch.float16, torch.bfloat16):
        kp, vp = _pages(layout, P, Hkv, ps, dtype, how)
        want = [kp.clone(memory_format=torch.contiguous_format),
                vp.clone(memory_format=torch.contiguous_format)]
        g = torch.Generator("cuda").manual_seed(T)
        qkv = torch.randn(T, 2 * Hkv + 1, 128, generator=g, device="cuda").to(dtype)
        qkv[0, 0, 0], qkv[-1, Hkv, 5] = float("nan"), float("inf")   # copied as they are
        k, v = qkv[:, :Hkv], qkv[:, Hkv:2 * Hkv]
        slot = torch.randperm(P * ps, generator=g, device="cuda")[:T]
        skip = torch.rand(T, generator=g, device="cuda") < 0.2
        slot = torch.where(skip, torch.tensor([-1, P * ps, 2 ** 40, -2 ** 40], device="cuda")
                           [torch.arange(T, device="cuda") % 4], slot)
        for t, s in enumerate(slot.tolist()):
            if 0 <= s < P * ps:
                for pages, x in zip(want, (k, v)):
                    if layout == "HND":
                        pages[s // ps, :, s % ps] = x[t]
                    else:
                        pages[s // ps, s % ps] = x[t]
        mab.paged_store(mab.PagedCache(kp, vp, layout), k, v, slot)
        torch.cuda.synchronize()
        assert torch.equal(kp.contiguous().view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(vp.contiguous().view(torch.int16), want[1].view(torch.int16))


def test_store_past_32_bit_offsets(cuda_lib):
    # 9 GB: the last page starts past 2^32 elements (a cache that is a slice of a larger tensor)
    P, Hkv, ps = 5, 8, 16
    page = Hkv * ps * 128
    step = 2 ** 30 + 2 * page
    base = torch.zeros(4 * step + 2 * page, dtype=torch.float16, device="cuda")
    shape, strides = (P, Hkv, ps, 128), (step, ps * 128, 128, 1)
    kp = torch.as_strided(base, shape, strides)
    vp = torch.as_strided(base, shape, strides, page)
    k = torch.randn(2, Hkv, 128, device="cuda").half()
    slot = torch.tensor([P * ps - 1, 0], device="cuda")
    mab.paged_store(mab.PagedCache(kp, vp), k, 2 * k, slot)
    torch.cuda.synchronize()
    assert torch.equal(kp[-1, :, -1], k[0]) and torch.equal(vp[-1, :, -1], 2 * k[0])
    assert torch.equal(kp[0, :, 0], k[1]) and torch.equal(vp[0, :, 0], 2 * k[1])
    assert int(torch.count_nonzero(base)) == 2 * int(torch.count_nonzero(k))


def test_more_returned_pages_than_an_int(cuda_lib):
    # lengths that claim 2^27 pages each: nothing past the stack or the rows is touched
    B, cols = 4096, 2 ** 20
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda").expand(B, cols)
    stack = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    with pytest.raises(mab.AttnError):   # rows may not overlap
        mab.paged_plan(_i32([2 ** 31 - 1] * B), _i32([-1] * B), stack[:10].contiguous(), _i32([0]),
                       table, 16, 0)
    table = torch.zeros(B, 64, dtype=torch.int32, device="cuda")
    guarded = torch.full((10 + 4096,), 9, dtype=torch.int32, device="cuda")
    plan = mab.paged_plan(_i32([2 ** 31 - 1] * B), _i32([-1] * B), guarded[:10], _i32([3]), table,
                          16, 0)
    torch.cuda.synchronize()
    assert int(plan.free_count) == 10 and plan.seqlen_k.sum() == 0
    assert guarded.tolist() == [9] * 3 + [0] * 7 + [9] * 4096


def test_host_threads_with_different_numbers_of_requests(cuda_lib):
    # both need more shared memory than a launch may use unasked, and the
    # smaller one must not lower the larger one's limit
    import threading
    sizes = (4096, 3500)
    errors = []

    def work(B):
        try:
            fresh, cached = _i32([1] * B), _i32([0] * B)
            stack, n = _i32(list(range(B))), _i32([B])
            table = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
            stream = torch.cuda.Stream()
            plan = mab.PagedPlan.empty(B, B, "cuda")
            torch.cuda.synchronize()
            for _ in range(1000):
                mab.paged_plan(cached, fresh, stack, n, table, 16, B, out=plan, stream=stream)
            stream.synchronize()
            assert plan.refused.item() == 0 and plan.free_count.item() == 0
        except Exception as e:  # noqa: BLE001 (reported below, from the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(B,)) for B in sizes for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


@pytest.mark.parametrize("T", [300, 5000])
def test_few_requests_with_many_pages(cuda_lib, T):
    # long requests that end, and long chunks, beside others: more pages and
    # tokens than the cluster has threads, and fewer
    ps, cols = 16, 3200
    cached = [50000, 0, 17, 40000, 16, 0, 33, 30000]
    fresh = [-1, T - 290, 1, -1, 200, 0, -1, 80]
    r = random.Random(5)
    pages = list(range(9000))
    r.shuffle(pages)
    table, at = [], 0
    for c in cached:
        h = -(-c // ps)
        table.append(pages[at:at + h] + [-5] * (cols - h))
        at += h
    stack = pages[at:] + [-3] * at
    _compare(cached, fresh, stack, len(pages) - at, table, ps, T)
    # the same with too few free pages for the last ones
    _compare(cached, fresh, stack, 1, table, ps, T)
