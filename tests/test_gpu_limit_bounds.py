"""Attention under key limits on the GPU, each element within a bound of its own
(limit_bounds.py), so that small gradients are checked beside large ones; and
beyond 128 tiles a head, where the tables come from launches of their own, the
causal mask's bits."""
import random

import pytest
import torch

import deterministic_attn_backward_gb300 as dab
import limit_bounds as lb
from gpu_common import case


def answers(prompt, lengths):
    return dab.prefix_limits([prompt] + lengths, [-1] + [0] * len(lengths))


def limits(name):
    rng = random.Random(11)
    if name == "prompt":
        return answers(700, [70, 1, 129, 33, 128, 200])
    if name == "short":          # up to 16 tiles: the forward reads the limits itself
        return answers(90, [50, 20, 1])
    if name == "groups":
        lengths, parents = [], []
        for _ in range(6):
            root = len(lengths)
            lengths += [rng.randint(300, 600)] + [rng.randint(1, 120) for _ in range(5)]
            parents += [-1] + [root] * 5
        return dab.prefix_limits(lengths, parents)
    if name == "any":
        return torch.tensor([rng.choice([0, rng.randrange(c, 700), 700]) for c in range(700)], dtype=torch.int32)
    if name == "many tiles":
        return dab.prefix_limits([900] + [400] * 30 + [3000] + [37] * 40, [-1] + [0] * 30 + [-1] + [31] * 40)
    raise ValueError(name)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name,heads", [("short", 3), ("prompt", 3), ("groups", 3), ("any", 2), ("many tiles", 1)])
def test_every_element(name, heads, d):
    limit = limits(name).cuda()
    S, scale = limit.numel(), d ** -0.5
    q, k, v, do = (t.cuda() for t in case(1, heads, S, d, 81))
    seen = lb.seen_under(limit)
    ws = dab.new_workspace(1, heads, S, d, "causal", "auto", "cuda", limit=True)
    o, lse = dab.attn_fwd(q, k, v, "causal", limit=limit, workspace=ws)
    assert dab.check_status(ws) == 0
    ref, bound = lb.forward(q, k, v, seen, scale)["o"]
    assert lb.tight(ref, bound) < 0.12 and lb.within(o, ref, bound)
    bounds = lb.backward(q, k, v, o, lse, do, seen, scale)
    for sched in ("descending_q", "serial", "atomic"):
        ws = dab.new_workspace(1, heads, S, d, "causal", sched, "cuda", limit=True)
        grads = dab.attn_bwd(q, k, v, o, lse, do, "causal", sched, limit=limit, workspace=ws)
        assert dab.check_status(ws) == 0
        for n, g in zip(("dq", "dk", "dv"), grads):
            ref, bound = bounds[n]
            assert lb.tight(ref, bound) < 0.12, n
            assert lb.within(g, ref, bound), (sched, n)


@pytest.mark.gpu
@pytest.mark.parametrize("S,d", [(128 * 128 + 1, 64), (128 * 131, 128), (17_380, 64)])
def test_limits_at_the_end_give_the_causal_bits_of_long_heads(S, d):
    assert S > 128 * 128
    q, k, v, do = (t.cuda() for t in case(1, 2, S, d, 82))
    limit = torch.full((S,), S, dtype=torch.int32, device="cuda")
    o, lse = dab.attn_fwd(q, k, v, "causal")
    o2, lse2 = dab.attn_fwd(q, k, v, "causal", limit=limit)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    for sched in ("serial", "descending_q"):
        plain = dab.attn_bwd(q, k, v, o, lse, do, "causal", sched)
        got = dab.attn_bwd(q, k, v, o, lse, do, "causal", sched, limit=limit)
        for a, b in zip(plain, got):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
