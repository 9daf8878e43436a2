"""Plain 64-bit attention for the tests: one head at a time from the
definition, with the bounds that the 16-bit operands allow.

Roundings of the kernels, per element, with u = eps / 2 of the 16-bit type
(a rounding is off by at most u times the value, or half the least subnormal):
  P  is rounded before O += P V and dV += P^T dO,
  dS is rounded before dQ += dS K and dK += dS^T Q,
  every 16-bit output is rounded once.
Everything else is fp32: a sum of 128 products is off by at most
128 * 2^-24 = 2^-17 of the sum of the absolute products, so a score is off by
at most ES = 2^-17 * scale * sum|q k| (plus 2^-21 for the exp2 and log2
approximations and the change of base), P by that relative amount, and
dP - Delta by 2^-17 (sum|dO v| + sum|dO o|).  fp32 sums over the keys or
queries of a row or column add their terms one by one in the matrix unit's
accumulator: n * 2^-24 of the sum of the absolute terms.
"""
from __future__ import annotations

import math

import torch


def u_of(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny_of(dtype) -> float:
    """Half the least subnormal: a rounding of a value below the normal range."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def window_first(rows, keys, window=None, first=0):
    """[n, l] visibility of key positions `keys` to query positions `rows`."""
    i, j = rows[:, None], keys[None, :]
    vis = j <= i
    if window is not None:
        vis = vis & ((i - j < window) | (j < first))
    return vis


def head_fwd(q, k, v, vis, sink, scale):
    """One head.  q [n, D], k, v [l, D] (16-bit), vis [n, l] bool, sink a float
    or None: (o, lse, bound of o, bound of lse) in float64."""
    dt = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    v = torch.where(vis.any(0)[:, None], v, 0.0)   # what nobody sees may be anything
    k = torch.where(vis.any(0)[:, None], k, 0.0)
    s = (q @ k.T) * scale
    es = 2.0 ** -17 * scale * (q.abs() @ k.abs().T) + 2.0 ** -21 * (1 + s.abs())
    s = torch.where(vis, s, -math.inf)
    es = torch.where(vis, es, 0.0)
    m = s.amax(1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, dtype=s.dtype,
                                                device=s.device)
    if sink is not None:
        m = m.clamp(min=float(sink))
    seen = m > -math.inf
    m = torch.where(seen, m, 0.0)
    e = torch.exp(s - m[:, None])
    l = e.sum(1)
    if sink is not None:
        l = l + torch.exp(float(sink) - m)
    ls = torch.where(seen, l, 1.0)
    p = e / ls[:, None]
    o = p @ v
    lse = torch.where(seen, m + torch.log(ls), math.inf)
    n = vis.sum(1)
    esm = es.amax(1) if s.shape[1] else torch.zeros_like(m)
    u = u_of(dt)
    absum = p @ v.abs()
    # P to 16 bits, the relative error of P (numerator and denominator), sums
    rel = u + 2 * esm + 2 * n * 2.0 ** -24 + 2.0 ** -20
    ob = absum * rel[:, None] + u * o.abs() + tiny_of(dt)
    # subnormal P: P is taken against a maximum with sum >= 2^-8 of the largest
    ob = ob + 2.0 ** 8 * tiny_of(dt) * (vis.double() @ v.abs()) / ls[:, None].clamp(min=1.0)
    lb = esm + n * 2.0 ** -24 + 2.0 ** -20 * (1 + lse.abs().nan_to_num(posinf=0.0))
    return o, lse, ob, lb


def head_bwd(q, k, v, o, dO, lse, vis, scale, compensated=False):
    """One query head from the given o and lse: dict of (value, bound)
    contributions dq, dk, dv (before the output's rounding) and delta."""
    dt = q.dtype
    q, k, v, o, dO, lse = (x.double() for x in (q, k, v, o, dO, lse))
    s = (q @ k.T) * scale
    es = 2.0 ** -17 * scale * (q.abs() @ k.abs().T) + 2.0 ** -21 * (1 + s.abs() + lse.abs()[:, None])
    p = torch.where(vis, torch.exp(torch.where(vis, s, 0.0) - lse[:, None]), 0.0)
    es = torch.where(vis, es, 0.0)
    delta = (dO * o).sum(1)
    dpa = dO.abs() @ v.abs().T + (dO * o).abs().sum(1)[:, None]
    ds = p * (dO @ v.T - delta[:, None])
    u, tiny = u_of(dt), tiny_of(dt)
    if compensated:   # high part + remainder: two roundings, the second of the remainder
        u = u * u
    ep = p * (u + es) + torch.where(vis, tiny, 0.0)
    eds = ds.abs() * (u + es) + p * 2.0 ** -17 * dpa + torch.where(vis, tiny, 0.0)
    # fp32 sums over the partners
    ep = ep + p * p.shape[0] * 2.0 ** -24
    edq = eds + ds.abs() * vis.shape[1] * 2.0 ** -24
    edk = eds + ds.abs() * vis.shape[0] * 2.0 ** -24
    return {"dq": (scale * (ds @ k), scale * (edq @ k.abs())),
            "dk": (scale * (ds.T @ q), scale * (edk.T @ q.abs())),
            "dv": (p.T @ dO, ep.T @ dO.abs()),
            "delta": delta, "delta_abs": (dO * o).abs().sum(1)}


def forward(q, k, v, vis, sink, scale):
    """BHSD tensors under vis(b) -> [Sq, Skv]: (o, lse, o bound, lse bound)."""
    B, Hq, Sq, D = q.shape
    g = Hq // k.shape[1]
    z = dict(dtype=torch.float64, device=q.device)
    o, ob = torch.zeros(B, Hq, Sq, D, **z), torch.zeros(B, Hq, Sq, D, **z)
    lse, lb = torch.zeros(B, Hq, Sq, **z), torch.zeros(B, Hq, Sq, **z)
    for b in range(B):
        for h in range(Hq):
            o[b, h], lse[b, h], ob[b, h], lb[b, h] = head_fwd(
                q[b, h], k[b, h // g], v[b, h // g], vis(b),
                None if sink is None else float(sink[h]), scale)
    return o, lse, ob, lb


def backward(q, k, v, o, dO, lse, vis, sink, scale, compensated=False):
    """BHSD tensors: {"dq": (value, bound), ...}, the output rounding included."""
    B, Hq, Sq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    z = dict(dtype=torch.float64, device=q.device)
    out = {n: [torch.zeros(t.shape, **z), torch.zeros(t.shape, **z)]
           for n, t in (("dq", q), ("dk", k), ("dv", v))}
    dsink = [torch.zeros(Hq, **z), torch.zeros(Hq, **z)]
    for b in range(B):
        for h in range(Hq):
            r = head_bwd(q[b, h], k[b, h // g], v[b, h // g], o[b, h], dO[b, h], lse[b, h],
                         vis(b), scale, compensated)
            for i in range(2):
                out["dq"][i][b, h] += r["dq"][i]
                out["dk"][i][b, h // g] += r["dk"][i]
                out["dv"][i][b, h // g] += r["dv"][i]
            if sink is not None:
                live = vis(b).any(1)
                w = torch.exp(float(sink[h]) - lse[b, h].double())
                w = torch.where(live, w, 0.0)
                dsink[0][h] -= (w * r["delta"]).sum()
                # fp32: Delta's sum of 128, exp of a difference, a sum over Sq rows
                dsink[1][h] += (w * r["delta_abs"]).sum() * (2.0 ** -16 + Sq * 2.0 ** -24) \
                    + (w * r["delta"].abs() * 2.0 ** -20 * (1 + lse[b, h].double().abs())).sum()
    u = u_of(q.dtype)
    res = {n: (x, e + u * x.abs() + tiny_of(q.dtype)) for n, (x, e) in out.items()}
    if sink is not None:
        res["dsink"] = tuple(dsink)
    return res


def check(name, got, value, bound):
    """Every element of `got` within `bound` of `value`; infinities equal."""
    g = got.double()
    assert g.shape == value.shape, (name, g.shape, value.shape)
    inf = torch.isinf(value)
    assert torch.equal(torch.where(inf, g, 0.0), torch.where(inf, value, 0.0)), name
    err = torch.where(inf, 0.0, g - value).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int((err / bound.clamp(min=1e-300)).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst at flat {i}: "
                             f"{g.flatten()[i]} for {value.flatten()[i]}, "
                             f"bound {bound.flatten()[i]:.3g}")
