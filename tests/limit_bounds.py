"""Attention under a mask in float64 beside how far the kernels' results may be from
it, element by element.

What the kernels round (2^-8 is half a step of bf16, 2^-24 of f32): P to bf16, and
dS = P (dP - D) to bf16 once more; the products' sums are f32; the result is bf16.
With terms t_i of an element's sum (P V, P dO, dS K or dS Q):

- The roundings are independent and of either sign, each at most r |t_i|, r = 2^-8
  for P and 2 * 2^-8 (1 + 2^-8) for dS.  Their sum passes 7 r sqrt(sum t_i^2) with
  probability 2 exp(-7^2 / 2) = 5e-11 (Hoeffding), and r sum |t_i| never.
- P's exponent is off by x: the score's sum of d products (2^-23 each, the tensor
  cores may cut off instead of rounding), the scaling and the offset (2^-24 of each
  magnitude, four of them) and 2^-21 for the exponential: x |t_i| each, all of
  one sign at worst.
- dP and D are sums of d exact products, off by d 2^-23 sum |dO V| and d 2^-24 sum
  |dO O|: together at most e, P e in dS.  Only here does an error not shrink
  with dS, which matters where dP and D agree (rows that see one key).
- Adding n terms in f32 is off by n 2^-24 of the running sum, at most 7 sqrt(sum
  t_i^2) as above.

D is taken from the rounded O and P from the rounded LSE that the backward is
given, so neither's own rounding counts."""
from __future__ import annotations

import torch

HALF = 2.0 ** -8


def _exponent(q, k, lse, scale):
    d = q.shape[-1]
    room = d * 2.0 ** -23 * scale * (q.abs() @ k.abs().mT).amax()
    most = torch.where(torch.isfinite(lse), lse.abs(), 0.0).amax()
    return float(2 * (room + 4 * 2.0 ** -24 * (2 * most + 1)) + 2.0 ** -21)


def _sum_bound(left, right, r, x, n):
    """Of left @ right, the terms' roundings r and exponents' x as above."""
    root = (left.square() @ right.square()).sqrt()
    total = left.abs() @ right.abs()
    return torch.minimum(7 * r * root, r * total) + x * total + n * 2.0 ** -24 * torch.minimum(7 * root, total)


def _rounded(ref, bound):
    return bound + HALF * (ref.abs() + bound) + 1e-30


def seen_under(limit):
    at = torch.arange(limit.numel(), device=limit.device)
    return (at[None, :] <= at[:, None]) & (at[:, None] < limit[None, :].long())


def forward(q, k, v, seen, scale):
    """{"o": (reference, bound)}; rows that see nothing are 0."""
    q, k, v = (t.double() for t in (q, k, v))
    s = (scale * q @ k.mT).masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.nan_to_num(torch.exp(s - lse[..., None]))
    o = p @ v
    x = 2 * _exponent(q, k, lse, scale)            # of P and of the sum it is divided by
    return {"o": (o, _rounded(o, _sum_bound(p, v, HALF, x, q.shape[-2])))}


def backward(q, k, v, o, lse, do, seen, scale):
    """{"dq": (reference, bound), "dk": ..., "dv": ...} for the o and lse given."""
    q, k, v, o, lse, do = (t.double() for t in (q, k, v, o, lse, do))
    d, n = q.shape[-1], q.shape[-2]
    p = torch.exp((scale * q @ k.mT - torch.where(lse == -torch.inf, torch.inf, lse)[..., None]))
    p = torch.where(seen, p, 0.0)
    ds = p * (do @ v.mT - (do * o).sum(-1, keepdim=True))
    e = float(d * 2.0 ** -23 * (do.abs() @ v.abs().mT).amax() + d * 2.0 ** -24 * (do * o).abs().sum(-1).amax())
    x = _exponent(q, k, lse, scale)
    r = 2 * HALF * (1 + HALF)
    out = {}
    for name, left, right, rest in (("dq", ds, k, p), ("dk", ds.mT, q, p.mT)):
        ref = scale * (left @ right)
        out[name] = (ref, _rounded(ref, scale * (_sum_bound(left, right, r, x, n) + e * (rest @ right.abs()))))
    dv = p.mT @ do
    out["dv"] = (dv, _rounded(dv, _sum_bound(p.mT, do, HALF, x, n)))
    return out


def within(got, ref, bound) -> bool:
    return bool(((got.double() - ref).abs() <= bound).all())


def tight(ref, bound) -> float:
    """The bound's share of the reference, as norms: a result of zeros is off by 1."""
    return float(bound.norm() / ref.norm())
