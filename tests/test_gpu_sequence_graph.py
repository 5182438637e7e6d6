"""Captured sequence operators and their workspaces: a graph's workspace is
its own, whatever is called or replayed beside it."""
import pytest
import torch

from deformable_convolution_amd import sequence

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def calls(seed, B, L, C=64):
    """Every operator that takes a workspace: attention's gradients, split attention, layer norm's gradients."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    q, k, v, g = (rand(B, L, 2, 64) for _ in range(4))
    cache = rand(1, 4096, 1, 64)
    x, dy = rand(B, C, L), rand(B, C, L)

    def call():
        out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
        grads = sequence.attention_backward(q, k, v, out, lse, g, causal=True)
        step = sequence.attention(q[:1, :1, :1], cache, cache)
        _, mean, rstd = sequence.layer_norm(x, with_stats=True)
        norm = sequence.layer_norm_backward(x, dy, mean, rstd)
        return [out, lse, *grads.values(), step, *norm.values()]

    return call


def captured(call, stream=None):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = call()
    return graph, got


def test_a_larger_call_after_the_capture():
    small, large = calls(1, 2, 130), calls(2, 8, 1100, C=512)
    want = [t.clone() for t in small()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        small()  # this stream's workspace is cached ahead of the capture
    torch.cuda.synchronize()
    graph, got = captured(small, side)
    with torch.cuda.stream(side):
        large()  # and replaced after it
    torch.cuda.synchronize()
    # what took over the memory that the larger call gave back, if any
    with torch.cuda.stream(side):
        others = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (1 << 10, 1 << 20, 1 << 20, 2 << 20, 8 << 20)]
    for _ in range(3):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all((t == 7).all() for t in others)
        large()
        torch.cuda.synchronize()


def test_two_graphs_at_once():
    made = [calls(3, 2, 700), calls(4, 2, 700)]
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


def test_a_workspace_given_is_used():
    call = calls(5, 2, 130)
    q = torch.randn((1, 1, 1, 64), device=DEV)
    cache = torch.randn((1, 4096, 1, 64), device=DEV)
    want = sequence.attention(q, cache, cache)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
    graph, got = captured(lambda: [sequence.attention(q, cache, cache, workspace=ws)])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and not (ws == 255).all()
    call()
