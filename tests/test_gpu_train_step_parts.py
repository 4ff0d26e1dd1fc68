"""The training step of test_gpu_train_step.py with each part checked on what the
step really handed it, so that the bounds are those of the part alone: the
attention element by element (limit_bounds.py), the table's gradient against
float64 sums of the step's own bf16 rows, the norm against that gradient, and the
clipped values against the norm in float64."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab
import limit_bounds as lb
from test_gpu_train_step import D, HEADS, ROWS, SCALE, WIDTH, Step, flat, heads, inputs

EPS = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [1, 2])
def test_the_parts_of_a_step(seed):
    ids, limit, table, upstream, other = inputs(seed)
    S = ids.numel()
    step = Step(S)
    o, norm, grad, rest = (t.clone() for t in step(ids, limit, table, upstream, other))
    # the same calls one by one: the step's bits, with what lies between them
    x = heads(dab.embed_fwd(ids, table, SCALE, dtype=torch.bfloat16))
    want = table[ids].double() * SCALE
    assert bool(((flat(x).double() - want).abs() <= want.abs() * (2.0 ** -8 * (1 + 2 * EPS) + 2 * EPS)).all())
    oh, lse = dab.attn_fwd(x, x, x, "causal", limit=limit)
    assert torch.equal(flat(oh), o)
    seen, do = lb.seen_under(limit), heads(upstream)
    assert lb.within(oh, *lb.forward(x, x, x, seen, D ** -0.5)["o"])
    grads = dab.attn_bwd(x, x, x, oh, lse, do, "causal", "auto", limit=limit)
    bounds = lb.backward(x, x, x, oh, lse, do, seen, D ** -0.5)
    for n, g in zip(("dq", "dk", "dv"), grads):
        assert lb.tight(*bounds[n]) < 0.12 and lb.within(g, *bounds[n]), n
    # dq + dk + dv: two f32 additions and a rounding to bf16
    dx = flat(sum(g.float() for g in grads).bfloat16()).contiguous()
    plain = dab.embed_bwd(ids, dx, ROWS, SCALE, dtype=torch.float32, padding=0)
    kept = dx.double() * (ids != 0)[:, None]
    zero = torch.zeros(ROWS, WIDTH, dtype=torch.float64, device="cuda")
    sums, mags = zero.index_add(0, ids, kept) * SCALE, zero.index_add(0, ids, kept.abs()) * SCALE
    count = torch.bincount(ids, minlength=ROWS).double()[:, None]
    room = (count + 3) * EPS * mags       # c - 1 additions, the product, SCALE in f32, the rounding, one to spare
    assert bool(((plain.double() - sums).abs() <= room).all())
    # the norm of exactly these: 12 * 2^-24 (test_gpu_grad_norm)
    exact = float((plain.double().square().sum() + other.double().square().sum()).sqrt())
    assert abs(float(norm) - exact) <= 12 * EPS * exact
    f = 1.0 / (exact + 1e-6)
    for got, before in ((grad, plain), (rest, other)):
        ref = before.double() * f
        assert bool(((got.double() - ref).abs() <= 16 * EPS * ref.abs() + 1e-40).all())
