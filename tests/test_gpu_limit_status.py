"""The status word of a forward under key limits: every CTA's waits read it, so it
is cleared by a launch ahead of the attention's, whatever the workspace held."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab
from gpu_common import case
from gpu_graph import captured_nodes


def call(S, tokens, d, ws):
    q, k, v, _ = (t.cuda() for t in case(1, 3, S, d, 61))
    limit = dab.prefix_limits([S // 2, S // 4, S - S // 2 - S // 4], [-1, 0, 0]).cuda()
    out, lse = torch.empty_like(q), torch.empty(1, 3, S, device="cuda")
    return lambda: dab.attn_fwd(q, k, v, "causal", limit=limit, tokens=tokens, workspace=ws, out=out, lse=lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,tokens", [(1, 1), (511, 511), (2048, 2048), (4096, 300), (2049, 2049)])
def test_the_status_is_cleared_ahead_of_the_attention(S, tokens, d):
    ws = dab.new_workspace(1, 3, S, d, "causal", "auto", "cuda", limit=True)
    kinds, roots = captured_nodes(call(S, tokens, d, ws))
    assert len(kinds) == 2 and kinds[-1] == "kernel" and roots == 1


@pytest.mark.gpu
@pytest.mark.parametrize("S", [130, 511, 2048, 2049])
def test_a_workspace_that_holds_an_error_changes_nothing(S):
    ws = dab.new_workspace(1, 3, S, 64, "causal", "auto", "cuda", limit=True)
    run = call(S, S, 64, ws)
    want = [t.clone() for t in run()]
    for _ in range(50):
        ws.fill_(0xFF)
        got = run()
        assert dab.check_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
