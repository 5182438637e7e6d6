"""Group norm and the gated recurrence captured into graphs, on other streams,
at once, and with workspaces: a graph's workspace is its own, whatever is
called or replayed beside it."""
import pytest
import torch

from deformable_convolution_amd import sequence

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def calls(seed, B, L, C=64, dtype=torch.float32):
    """A norm with its gradients over samples that are held and over samples in parts, a recurrence with its gradients
    in several segments and a single position."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    x, gate, go, w, b = rand(B, L, C), rand(B, L, C), rand(B, L, C), rand(C), rand(C)
    few, state = rand(B, C), torch.randn((B, C), generator=gen, device=DEV)

    def call():
        got = []
        for t, g in ((x, 1), (few, 4)):
            y, mean, rstd = sequence.group_norm(t, g, w, b, activation="silu", with_stats=True)
            grads = sequence.group_norm_backward(t, g, go if t is x else few, mean, rstd, w, b, "silu")
            got += [y, mean, rstd, *grads.values()]
        y, last, states = sequence.gated_recurrence(x, gate, state, blend=True, with_states=True)
        grads = sequence.gated_recurrence_backward(x, gate, states, go, last, blend=True)
        step = sequence.gated_recurrence(x[:, :1], gate[:, :1], state)
        return got + [y, last, states, *grads.values(), *step]

    return call


def captured(call, stream=None):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = call()
    return graph, got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_replays_between_eager_calls(dtype):
    small, large = calls(1, 2, 3000, dtype=dtype), calls(2, 3, 9000, C=96, dtype=dtype)
    want = [t.clone() for t in small()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        small()  # this stream's workspace is cached ahead of the capture
    torch.cuda.synchronize()
    graph, got = captured(small, side)
    with torch.cuda.stream(side):
        large()  # and replaced after it
    torch.cuda.synchronize()
    for _ in range(4):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        large()
        assert all(torch.equal(a, b) for a, b in zip(want, small()))
        torch.cuda.synchronize()


def test_two_graphs_at_once():
    made = [calls(3, 2, 3000), calls(4, 2, 3000)]
    want = [[t.clone() for t in call()] for call in made]
    torch.cuda.synchronize()
    graphs = [captured(call) for call in made]  # both on torch's own capture stream
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for _, got in graphs:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, got), ref in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_streams_at_once():
    made = [calls(5, 2, 3000), calls(6, 1, 7000)]
    want = [[t.clone() for t in call()] for call in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for call, stream in zip(made, streams):
            with torch.cuda.stream(stream):
                got.append(call())
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
