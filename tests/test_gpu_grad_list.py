"""A gradient list's workspace: its status word, and the streams that use it."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[], [0], [1000, 3], [40_000] * 70, [5] * 2100])
def test_every_call_leaves_the_status_clear(sizes):
    grads = dab.GradList([torch.ones(n, device="cuda") for n in sizes])
    given = torch.tensor(2.0, device="cuda")
    for call in (lambda: dab.grad_norm(grads), lambda: dab.clip_grads(grads, 1.0),
                 lambda: dab.clip_grads(grads, 1.0, norm=given)):
        grads.workspace.fill_(0xFF)
        call()
        assert dab.check_status(grads.workspace) == 0
