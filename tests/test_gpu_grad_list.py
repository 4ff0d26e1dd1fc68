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


@pytest.mark.gpu
def test_a_workspace_used_on_another_stream_is_not_handed_out_meanwhile():
    """A list is made on one stream, used on another and dropped while that one is
    still busy: its workspace stays taken until the sums are done."""
    g = torch.full((30_000_000,), 2.0, device="cuda")
    side = torch.cuda.Stream()
    grads = dab.GradList([g])
    size, at = grads.workspace.numel(), grads.workspace.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                     # some 50 ms
        norm = dab.clip_grads(grads, 1.0)
        busy = torch.cuda.Event()
        busy.record(side)
    del grads
    taken = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not busy.query(), "the other stream had already ended"
    assert all(t.data_ptr() != at for t in taken)
    side.synchronize()
    assert abs(float(norm) - 2.0 * 30_000_000 ** 0.5) < 0.01
    # from the stream it was made on, it is free again as soon as it is dropped
    grads = dab.GradList([g])
    at = grads.workspace.data_ptr()
    dab.clip_grads(grads, 1.0)
    del grads
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() == at


@pytest.mark.gpu
def test_a_list_made_beside_a_capture():
    """A captured call on another stream than the list's: it may be dropped after the graph."""
    g = torch.full((5000,), 2.0, device="cuda")
    grads = dab.GradList([g])
    dab.clip_grads(grads, 1e9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = dab.clip_grads(grads, 1e9)
    for k in (3.0, 1.0):
        g.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - k * 5000 ** 0.5) < 1e-3
    del graph, grads
    torch.cuda.synchronize()
    assert torch.zeros(1 << 16, device="cuda").sum() == 0
