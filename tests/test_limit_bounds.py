"""The element-by-element bounds of the attention tests, on the CPU: a float32
computation with the kernels' roundings stays within them, and mistakes do not."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab
import limit_bounds as lb


def bf(t):
    return t.bfloat16().float()


def rounded(q, k, v, do, seen, scale):
    """o, lse, dq, dk, dv in float32 with P, dS and the results in bf16."""
    q, k, v, do = (t.float() for t in (q, k, v, do))
    s = (scale * q @ k.mT).masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, -1)
    top = torch.nan_to_num(s.amax(-1, keepdim=True), neginf=0.0)
    p = torch.exp(s - top)
    o = torch.nan_to_num(bf(p) @ v / p.sum(-1, keepdim=True)).bfloat16()
    p = bf(torch.where(seen, torch.exp(s - torch.where(lse == -torch.inf, torch.inf, lse)[..., None]), 0.0))
    ds = bf(p * (do @ v.mT - (do * o.float()).sum(-1, keepdim=True)))
    return {"o": o, "lse": lse, "dq": (scale * ds @ k).bfloat16(), "dk": (scale * ds.mT @ q).bfloat16(),
            "dv": (p.mT @ do).bfloat16()}


CASES = {"causal": [900], "answers": [400] + [70] * 6, "groups": [300, 100, 90, 200, 150]}
PARENTS = {"causal": [-1], "answers": [-1] + [0] * 6, "groups": [-1, 0, 0, -1, 3]}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", CASES)
def test_bounds_hold_for_the_roundings_and_not_for_mistakes(name, d):
    g = torch.Generator().manual_seed(5)
    limit = dab.prefix_limits(CASES[name], PARENTS[name])
    S, scale = limit.numel(), d ** -0.5
    q, k, v, do = (torch.randn(1, 2, S, d, generator=g).bfloat16() for _ in range(4))
    seen = lb.seen_under(limit)
    got = rounded(q, k, v, do, seen, scale)
    bounds = {**lb.forward(q, k, v, seen, scale), **lb.backward(q, k, v, got["o"], got["lse"], do, seen, scale)}
    for n, (ref, bound) in bounds.items():
        assert lb.within(got[n], ref, bound), n
        assert lb.tight(ref, bound) < 0.12, n
        assert not lb.within(torch.zeros_like(ref), ref, bound), n
        assert not lb.within(0.9 * ref, ref, bound), n
    # one 128-key tile hidden from one 128-query tile
    part = seen.clone()
    part[256:384, 128:256] = False
    wrong = rounded(q, k, v, do, part, scale)
    assert not lb.within(wrong["o"], *bounds["o"])
    wrong = lb.backward(q, k, v, got["o"], got["lse"], do, part, scale)
    assert not any(lb.within(wrong[n][0], *bounds[n]) for n in ("dq", "dk", "dv"))
    # one pair too many
    more = seen.clone()
    more[S - 1, :] = True
    more[0, 1] = True
    wrong = lb.backward(q, k, v, got["o"], got["lse"], do, more, scale)
    assert not lb.within(wrong["dv"][0], *bounds["dv"])
