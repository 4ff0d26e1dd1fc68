"""Host tensors given to the training step's operators: a call uses the values that
they hold when it is made, also when the copy waits behind other work and the
caller refills its pinned buffer at once.  A captured call reads it in each replay."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab
from gpu_common import case

S, WIDTH, ROWS = 300, 64, 50


def pinned(t):
    return t.cpu().pin_memory()


def made():
    """{name: (host tensors, call of them)}; every call is made of copies on the device once."""
    q, k, v, do = case(1, 2, S, 64, 71)
    dev = [t.cuda() for t in (q, k, v, do)]
    limit = dab.prefix_limits([100, 120, 80], [-1, 0, 0])
    ids = torch.randint(ROWS, (S,), generator=torch.Generator().manual_seed(1))
    table = torch.randn(ROWS, WIDTH, device="cuda")
    dout = torch.randn(S, WIDTH, device="cuda")
    o, lse = dab.attn_fwd(*dev[:3], "causal", limit=limit.cuda())
    return {
        "embed_fwd": ([ids], lambda i: [dab.embed_fwd(i, table)]),
        "embed_fwd int32": ([ids.int()], lambda i: [dab.embed_fwd(i, table)]),
        "embed_bwd": ([ids], lambda i: [dab.embed_bwd(i, dout, ROWS)]),
        "embed_bwd strided": ([torch.stack([ids, ids], 1)], lambda i: [dab.embed_bwd(i[:, 0], dout, ROWS)]),
        "attn_fwd limit": ([limit], lambda m: dab.attn_fwd(*dev[:3], "causal", limit=m)),
        "attn_fwd all": ([limit.long(), q, k, v], lambda m, *x: dab.attn_fwd(*x, "causal", limit=m)),
        "attn_bwd limit": ([limit, lse.cpu()], lambda m, x: dab.attn_bwd(*dev[:3], o, x, dev[3], "causal", "auto", limit=m)),
    }


NAMES = ["embed_fwd", "embed_fwd int32", "embed_bwd", "embed_bwd strided", "attn_fwd limit", "attn_fwd all",
         "attn_bwd limit"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_pinned_buffer_may_be_refilled_after_the_call(name):
    host, call = made()[name]
    want = call(*[t.cuda() for t in host])
    call(*[pinned(t) for t in host])                    # the pinned memory that the calls need is there
    held = [pinned(t) for t in host]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                      # some 50 ms
    done = torch.cuda.Event()
    got = call(*held)
    done.record()
    for t in held:
        t.zero_()
    assert not done.query(), "the call waited for the work ahead of it"
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_a_captured_call_reads_the_pinned_buffer_in_each_replay():
    ids = torch.arange(40)
    table = torch.randn(ROWS, WIDTH, device="cuda")
    held = ids.pin_memory()
    dab.embed_fwd(held, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dab.embed_fwd(held, table)
    for shift in (3, 7):
        held.copy_((ids + shift) % ROWS)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, table[((ids + shift) % ROWS).cuda()])
