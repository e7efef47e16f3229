"""A training step captured in a CUDA graph while something holds what adds to its
leaves' gradients: refused where that was made on the default stream (torch would end
the process), captured where it was not."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
K = 3


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(seed=0, T=40, n=8, d=144, d_ff=80):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [r(T, d).requires_grad_(), (r(n, d) / d ** 0.5).requires_grad_(), (r(n, 2 * d_ff, d) / d ** 0.5).requires_grad_(),
            (r(n, d, d_ff) / d_ff ** 0.5).requires_grad_()], r(T, d)


def fresh(leaves):
    return [p.detach().clone().requires_grad_() for p in leaves]


def capture(ex, leaves, d_out, stream):
    """(graph, its gradients), by backward(), which adds to the leaves."""
    for p in leaves:
        p.grad = None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ex.moe_train_f8(*leaves, K).backward(d_out)
    return graph, [p.grad for p in leaves]


def refused(ex, leaves, d_out):
    with pytest.raises(RuntimeError, match="no eager graph holds"):
        capture(ex, leaves, d_out, torch.cuda.Stream())


def holds(ex, leaves, d_out):
    """A capture's replays give the eager step's bits."""
    want = fresh(leaves)
    ex.moe_train_f8(*want, K).backward(d_out)
    graph, grads = capture(ex, leaves, d_out, torch.cuda.Stream())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.grad) for a, b in zip(grads, want))
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


@pytest.mark.parametrize("which", range(4))
def test_a_graph_that_torch_alone_has_built(ex, which):
    leaves, d_out = inputs()
    living = leaves[which] * 2
    refused(ex, leaves, d_out)
    refused(ex, leaves, d_out)
    del living
    holds(ex, leaves, d_out)


def test_every_part_looks(ex):
    leaves, _ = inputs()
    x, router, gate_up, _ = leaves
    logits = torch.randn(40, 8, device="cuda").requires_grad_()
    with torch.no_grad():
        idx, w = ex.top_k(logits, K)
        xs, offsets, place = ex.dispatch(x, idx, 8)
    w.requires_grad_()
    calls = [(logits, lambda: ex.top_k(logits, K)), (logits, lambda: ex.route(logits, K)), (x, lambda: ex.dispatch(x, idx, 8)),
             (gate_up, lambda: ex.experts_f8(xs, gate_up, offsets)), (w, lambda: ex.combine(xs, place, w))]
    for leaf, call in calls:
        living = leaf * 2
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="no eager graph holds"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
                call()
        del living
        living = call()  # a graph of this call's own
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="no eager graph holds"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
                call()
        del living
    assert ex.smoe.smoe_last_device_status() == ex.smoe.SMOE_OK


def test_what_keeps_the_node_on_the_default_stream(ex):
    """Refused for as long as it is kept, whatever ran in between."""
    leaves, d_out = inputs(1)
    kept = torch.autograd.graph.get_gradient_edge(leaves[2])
    refused(ex, leaves, d_out)
    ex.moe_train_f8(*leaves, K).backward(d_out)
    refused(ex, leaves, d_out)
    del kept
    holds(ex, leaves, d_out)


def test_a_living_graph_of_another_stream(ex):
    """The warm-up's output is still there, as in a loop that has not left its scope."""
    leaves, d_out = inputs(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        living = ex.moe_train_f8(*leaves, K)
        living.backward(d_out)
    torch.cuda.synchronize()
    holds(ex, leaves, d_out)
    assert living.requires_grad


def test_what_keeps_the_node_on_another_stream(ex):
    """Its stream is not known until a backward pass has run through it; then it is, and
    a capture goes through."""
    leaves, d_out = inputs(3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kept = [torch.autograd.graph.get_gradient_edge(p) for p in leaves]
    refused(ex, leaves, d_out)
    with torch.cuda.stream(s):
        ex.moe_train_f8(*leaves, K).backward(d_out)
    torch.cuda.synchronize()
    holds(ex, leaves, d_out)
    holds(ex, leaves, d_out)
    assert len(kept) == 4
