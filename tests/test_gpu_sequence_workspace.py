"""The sequence operators' workspace argument."""
import pytest
import torch

from deformable_convolution_amd import dc1d, sequence

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def calls():
    gen = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    q, k, v, g = rand(1, 1, 2, 64), rand(1, 4096, 1, 64), rand(1, 4096, 1, 64), rand(1, 1, 2, 64)
    out, lse = sequence.attention(q, k, v, with_lse=True)
    x, dy = rand(2, 64, 40), rand(2, 64, 40)
    _, mean, rstd = sequence.layer_norm(x, with_stats=True)
    return [lambda ws: [sequence.attention(q, k, v, workspace=ws)],
            lambda ws: list(sequence.attention_backward(q, k, v, out, lse, g, workspace=ws).values()),
            lambda ws: list(sequence.layer_norm_backward(x, dy, mean, rstd, workspace=ws).values())]


def test_views_that_hold_less_memory_than_elements_are_refused():
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    some = torch.full((1 << 24,), 7, dtype=torch.uint8, device=DEV)
    for call in calls():
        for ws in (one.expand(1 << 24), some[:1 << 12].view(1, -1).expand(1 << 12, -1), some[::2], some.view(1 << 12, -1)[:, :1 << 11]):
            with pytest.raises(ValueError):
                call(ws)
    torch.cuda.synchronize()
    assert (some == 7).all()


def test_any_contiguous_tensor_serves():
    for call in calls():
        want = call(None)
        for ws in (torch.empty(1 << 24, dtype=torch.uint8, device=DEV), torch.empty((64, 1 << 16), device=DEV),
                   torch.empty(1 << 24, dtype=torch.bfloat16, device=DEV)[1 << 20:]):
            assert all(torch.equal(a, b) for a, b in zip(call(ws), want))
        with pytest.raises(dc1d.Dc1dValueError) as e:
            call(torch.empty(16, dtype=torch.uint8, device=DEV))
        assert e.value.status == dc1d.ERR_WORKSPACE
