"""The attention's calls on a given stream: what they allocate belongs to it, and other streams' memory
does not become theirs; workspaces and inputs that lie elsewhere, and a second gradient, are refused."""
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


def test_workspaces_elsewhere_are_refused():
    for ws in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            fa._workspace(ws, 100, torch.device("cuda", 0))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(window=100, sinks=4)])
def test_a_given_stream_owns_what_the_call_allocates(kw):
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(1500, h, 128, generator=g).bfloat16().cuda() for h in (4, 2, 2, 4))
    kw = dict(kw, causal=True, batch=1)
    o, lse = fa.forward(q, k, v, **kw)
    want = (o, lse) + fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    here = torch.cuda.memory_stats()["allocated_bytes.all.current"]
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(2e7))  # the calls wait behind this, while the host goes on
    held, junk = [], []
    for s in (side, side.cuda_stream):
        x = fa.forward(q, k, v, stream=s, **kw)
        held.append(x + fa.backward(q, k, v, x[0], do, x[1], deterministic=True, stream=s, **kw))
        # what this stream allocates now is none of the call's workspaces
        junk += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 14, 1 << 20, 4 << 20, 4 << 20)]
        junk = junk[-4:]
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocated_bytes.all.current"] > here
    for got in held:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_inputs_elsewhere_are_refused():
    q = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="CUDA device"):
        fa.forward(q, q.cpu(), q, batch=1)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.forward(q, q, q, batch=1, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(window=5, sinks=1)])
def test_a_gradient_of_gradients_is_refused(kw):
    """The kernels' gradients are cut off from the inputs: what depends on both must not lose a part."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(30, 2, 64, generator=g).bfloat16().cuda().requires_grad_() for _ in range(3))
    o = fa.attention(q, k, v, causal=True, batch=1, **kw)
    dq, = torch.autograd.grad(o.float().square().sum(), q, create_graph=True)
    assert torch.isfinite(dq).all()
    with pytest.raises(RuntimeError, match="differentiable once"):
        (dq.float().sum() + q.float().sum()).backward()
