"""The 8-bit cache in plain form: codes as the numbers they stand for, scales as
exponents, everything from the definitions in 64 bits.

Blocks of tokens of a kv head share a scale 2^e; value = code * 2^e.  A run of new
rows that begins at a block's row 0 begins the block anew; one that begins at row
r0 > 0 keeps the rows below r0 and takes the larger of the two exponents, the
earlier codes rounded again in units of it."""
from __future__ import annotations

import math

import torch

TOP = {"e4m3": 448.0, "i8": 127.0}
LEAST = {("e4m3", torch.float16): -15, ("i8", torch.float16): -24,
         ("e4m3", torch.bfloat16): -110, ("i8", torch.bfloat16): -110}
TYPES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def e4m3_numbers():
    """The non-negative e4m3 numbers in the order of their codes 0 .. 126."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def nearest(kind, x, limit):
    """The nearest code numbers of x (ties to even codes), at most `limit`."""
    if kind == "i8":
        lim = math.floor(min(limit, 127.0))
        return torch.round(x).clamp(-lim, lim)
    t = e4m3_numbers().to(x.device)
    t = t[t <= limit]
    a = x.abs().contiguous()
    hi = torch.searchsorted(t, a).clamp(max=t.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = a - t[lo], t[hi] - a
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return torch.where(x < 0, -t[pick], t[pick])


def exponent(kind, dtype, amax):
    """The least e with amax <= TOP 2^e, held to the type's least."""
    out = torch.empty(amax.shape, dtype=torch.int64)
    for i, a in enumerate(amax.flatten().tolist()):
        e = -200 if a == 0 else math.frexp(a)[1] - 20
        while a > TOP[kind] * 2.0 ** e:
            e += 1
        out.view(-1)[i] = max(e, LEAST[kind, dtype])
    return out


class Cache64:
    """num [pages, ps, Hkv, 128], the code numbers; exp [pages, Hkv, blocks], None
    where not finite (999)."""
    BAD = 999

    def __init__(self, P, Hkv, ps, block, kind, dtype):
        self.ps, self.block, self.kind, self.dtype = ps, block, kind, dtype
        self.num = torch.zeros(P, ps, Hkv, 128, dtype=torch.float64)
        self.exp = torch.zeros(P, Hkv, ps // block, dtype=torch.int64)

    def store(self, x, slots):
        """x [T, Hkv, 128]; slots a list."""
        T, blk, ps = len(slots), self.block, self.ps
        x = x.double().cpu()
        big = torch.finfo(self.dtype).max
        t = 0
        while t < T:
            n = 1
            if not 0 <= slots[t] < self.num.shape[0] * ps:
                t += 1
                continue
            while t + n < T and slots[t + n] == slots[t] + n and \
                    slots[t + n] // blk == slots[t] // blk:
                n += 1
            page, row = divmod(slots[t], ps)
            at, r0 = row // blk, row % blk
            rows = x[t:t + n]
            fine = torch.isfinite(rows).all(2).all(0)          # [Hkv]
            e = exponent(self.kind, self.dtype, rows.abs().amax((0, 2)).nan_to_num(0, 0, 0))
            e = torch.where(fine, e, self.BAD)
            had = self.exp[page, :, at].clone()
            if r0 > 0:
                e = torch.maximum(e, had)
            for h in range(x.shape[1]):
                eh, hh = int(e[h]), int(had[h])
                if eh == self.BAD:
                    continue
                unit = 2.0 ** eh
                if r0 > 0 and eh > hh:
                    old = self.num[page, row - r0:row, h]
                    self.num[page, row - r0:row, h] = nearest(self.kind, old * 2.0 ** (hh - eh),
                                                              TOP[self.kind])
                self.num[page, row:row + n, h] = nearest(
                    self.kind, rows[:, h] / unit, min(TOP[self.kind], big / unit))
            self.exp[page, :, at] = e
            t += n

    def values(self, slots):
        """[n, Hkv, 128] values of the slots in 64 bits."""
        s = torch.as_tensor(slots)
        page, row = s // self.ps, s % self.ps
        e = self.exp[page, :, row // self.block]
        v = self.num[page, row] * torch.exp2(e.clamp(max=500).double())[..., None]
        return torch.where((e == self.BAD)[..., None], math.nan, v)

    def codes(self, layout):
        """Pages as a tensor of codes."""
        c = self.num if layout == "NHD" else self.num.transpose(1, 2)
        return c.contiguous().float().to(TYPES[self.kind])

    def bytes(self):
        return torch.where(self.exp == self.BAD, 255, self.exp + 127).to(torch.uint8)


def make(cache_k, cache_v, layout="HND", device="cuda"):
    """The binding's cache of two plain ones."""
    from masked_attention_backward_gb300 import binding as mab
    return mab.PagedCache8(cache_k.codes(layout).to(device), cache_v.codes(layout).to(device),
                           cache_k.bytes().to(device), cache_v.bytes().to(device),
                           cache_k.dtype, layout)
